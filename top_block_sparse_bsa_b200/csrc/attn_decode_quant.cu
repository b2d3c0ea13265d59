// attn_decode_quant.cu -- decode attention over the quantised paged cache
// (quant_cache.cu): one query token per sequence, each sequence its own
// length, over the kept blocks of a list or over every block.
//
// Formula.  A key is K_t 2^a_t, a value V_t 2^b_t (K, V rows of e4m3 codes,
// a, b the row's exponents).  With x_t = (q . K_t) 2^a_t scale log2(e) and
// y_t = x_t + b_t, any reference M >= about max y:
//   w_t = 2^(y_t - M),  O = sum w_t V_t,  l = sum w_t 2^-b_t,  o = O / l,
// so the value's exponent rides in the softmax weight and the matrix product
// takes the codes as they are.  lse = ln2 (M + log2 l).
//
// Bound: memory.  A key and its value are 2 (d + 1) bytes and 4 d operations
// for each of at most 16 heads; the cache's own bytes, read once per KV head
// for all its query heads, are the floor.  So the design keeps loads in
// flight and spends few instructions a byte:
//   - a warp takes 16 keys at a time, straight from memory into registers as
//     16-byte pieces: no shared-memory stage, no barrier, no block-wide wait in
//     the loop.  The next 16 keys are loaded while these keys' weights and
//     product are formed, the next values behind them.
//   - the codes become fp16 pairs by one conversion each (exact), and the
//     products run on m16n8k16 matrix instructions with the keys (then the
//     channels) as the 16 rows and eight query heads as the 8 columns.  The
//     order of the contracted index is free as long as both operands agree,
//     so each lane's share is whatever its 16-byte loads bring: channels for
//     q . K; for V, lanes pair two keys' bytes and number the channels as they
//     hold them.  Tensor-memory instructions would need the codes split from
//     their rows' exponents across lanes and a block-wide exchange of maxima
//     for every 128 keys, at twice the keys a second of the bf16 kernel, for
//     a part that is not the bound.
//   - M moves only when some y passes it by 2^7 (one vote a step; M starts at
//     the first maximum): w is scaled by 2^8, so it stays within fp16 and keeps
//     its 11 bits down to 2^-22 of the largest.
// w is rounded to fp16 for the product (at most 2^-11 of w); l sums it in fp32
// unrounded; logits, O and l are fp32.
//
// Work split: the rows' list positions are laid end to end, each sequence
// with the blocks it has, and cut into equal ranges, one per block of
// threads.  A range that holds a whole row writes its output; a row cut by
// range borders leaves one partial record (M, l, O) per range, at most two a
// block, and the second kernel joins them.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace bsa {
namespace qdecode {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kCtasPerSm = 2;
constexpr float kLift = 8.0f;        // weights are 2^(y - M + 8)
constexpr float kHeadroom = 7.0f;    // M moves when y > M + 7: weights stay below 2^15

__device__ __forceinline__ uint32_t cvt_e4m3x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// Ranges that `total` positions are cut into: none is empty.
__device__ __forceinline__ int ranges(int64_t total, int ctas) {
  return static_cast<int>(min(static_cast<int64_t>(ctas), total));
}

// First block of threads whose range [c total / C, (c+1) total / C) holds x.
__device__ __forceinline__ int cta_of(int64_t x, int64_t total, int C) {
  return static_cast<int>(((x + 1) * C + total - 1) / total) - 1;
}

// pre[b] = list positions of the sequences before b (of one KV head), b <= B:
// from a list every sequence has list_len positions, without one as many as
// it has blocks.
__device__ __forceinline__ void plan_positions(const QuantDecodeArgs& p, int* pre, int* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + tid;
    int w = 0;
    if (b < p.B) {
      const int len = p.lens ? min(max(p.lens[b], 0), p.nb * 64) : p.nb * 64;
      w = p.idx ? p.list_len : (len + 63) >> 6;
    }
    int incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int before = base, all = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) before += warp_sums[k];
      all += warp_sums[k];
    }
    if (b < p.B) pre[b] = before + incl - w;
    base += all;
    __syncthreads();
  }
  if (tid == 0) pre[p.B] = base;
  __syncthreads();
}

template <int D>
struct Shared {
  float o[kWarps][8][D + 4];
  float m[kWarps][8], l[kWarps][8];
  int warp_sums[kWarps];
};

// Where channel pair (r * D/8 + 2 mb) of a head is kept in Shared::o: the
// pairs of lane r are turned by r/2, so that a warp's stores fill the banks.
template <int D>
__device__ __forceinline__ int pair_at(int r, int mb) {
  return r * (D / 8) + 2 * ((mb + (r >> 1)) & (D / 16 - 1));
}

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_kernel(const QuantDecodeArgs p) {
  constexpr int KH = D / 64;        // 64-byte halves of a row
  constexpr int KS = D / 16;        // k-steps of q . K
  constexpr int MB = D / 16;        // 16-channel row blocks of O
  constexpr int VW = D / 32;        // 32-bit words of a V row per lane
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared<D>& sh = *reinterpret_cast<Shared<D>*>(smem_raw);
  int* pre = reinterpret_cast<int*>(smem_raw + sizeof(Shared<D>));
  griddep_wait();   // lists, lengths and the cache come from the kernels launched before
  plan_positions(p, pre, sh.warp_sums);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= p.B; b += kThreads) p.pre[b] = pre[b];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int G = p.Hq / p.Hkv;
  const int sets = (G + 7) / 8;                 // warps split into sets of eight query heads each
  const int per_set = kWarps / sets;
  const int set = warp / per_set, wi = warp % per_set;
  const int64_t total = static_cast<int64_t>(pre[p.B]) * p.Hkv;
  const int C = ranges(total, gridDim.x);
  if (static_cast<int>(blockIdx.x) >= C) return;
  int64_t x = blockIdx.x * total / C;
  const int64_t hi = (blockIdx.x + 1) * total / C;
  int b = 0;
  if (x < hi) {   // the sequence of position x: the last b with pre[b] * Hkv <= x
    int lo_b = 0, hi_b = p.B;
    while (hi_b - lo_b > 1) {
      const int mid = (lo_b + hi_b) / 2;
      if (static_cast<int64_t>(pre[mid]) * p.Hkv <= x) lo_b = mid; else hi_b = mid;
    }
    b = lo_b;
  }
  while (x < hi) {
    const int w = pre[b + 1] - pre[b];
    const int64_t seq0 = static_cast<int64_t>(pre[b]) * p.Hkv;
    if (w == 0 || x >= seq0 + static_cast<int64_t>(w) * p.Hkv) {
      ++b;
      continue;
    }
    const int g = static_cast<int>((x - seq0) / w);
    const int64_t row0 = seq0 + static_cast<int64_t>(g) * w;     // the row's first position
    const int t0 = static_cast<int>(x - row0);
    const int t1 = static_cast<int>(min(hi - row0, static_cast<int64_t>(w)));
    x = row0 + t1;
    const int bg = b * p.Hkv + g;
    const int len = p.lens ? min(max(p.lens[b], 0), p.nb * 64) : p.nb * 64;
    const int* list = p.idx ? p.idx + static_cast<int64_t>(bg) * p.list_len : nullptr;
    const int* table = p.table + static_cast<int64_t>(b) * p.table_stride;

    // ---- the query heads of this warp's set, scaled by a power of two into fp16
    uint32_t qf[KS][2];
    float qs[2];        // logit factors of heads 2c, 2c+1 of the set
    {
      const int h = set * 8 + r;
      uint32_t raw[KS][2];
      float amax = 0.0f;
      const __nv_bfloat16* qrow = p.q + (static_cast<int64_t>(b) * p.Hq + g * G + h) * D;
#pragma unroll
      for (int hf = 0; hf < KH; ++hf)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (h < G) v = __ldg(reinterpret_cast<const uint4*>(qrow + hf * 64 + c * 16 + 8 * i));
          raw[hf * 4 + 2 * i][0] = v.x;
          raw[hf * 4 + 2 * i][1] = v.y;
          raw[hf * 4 + 2 * i + 1][0] = v.z;
          raw[hf * 4 + 2 * i + 1][1] = v.w;
        }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(raw[k][i] << 16)),
                                   fabsf(__uint_as_float(raw[k][i] & 0xFFFF0000u))));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // the head's largest value goes to [2^10, 2^11): smaller ones keep their eight bits down to 2^-25 of it
      const int E = max(static_cast<int>(__float_as_uint(amax) >> 23), 11);
      const float up = __uint_as_float(static_cast<uint32_t>(264 - E) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qf[k][i] = pack_f16x2(__uint_as_float(raw[k][i] << 16) * up, __uint_as_float(raw[k][i] & 0xFFFF0000u) * up);
      const float down = __uint_as_float(static_cast<uint32_t>(E - 10) << 23) * p.scale_log2;
      qs[0] = __shfl_sync(0xffffffffu, down, (2 * c) * 4);
      qs[1] = __shfl_sync(0xffffffffu, down, (2 * c + 1) * 4);
    }

    float M[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    float O[MB][4];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) O[m][i] = 0.0f;

    // ---- chunks of 16 keys: this warp's are wi, wi + per_set, ...; 32 of them are looked up at once, one a lane
    const int chunks = 4 * (t1 - t0);
    int base = wi - 32 * per_set;        // first chunk of the batch held
    unsigned left = 0u;                  // lanes whose chunk is still to be taken
    int my_row = 0, my_n = 0;            // the lane's chunk: row of 16 in the pools, keys that count
    int row = 0, n = 0;                  // the chunk that the loads below are for
    auto next = [&]() -> bool {
      while (left == 0u) {
        base += 32 * per_set;
        if (base >= chunks) return false;
        const int u = base + lane * per_set;
        my_n = 0;
        if (u < chunks) {
          const int t = t0 + (u >> 2);
          const int blk = list ? __ldg(list + t) : t;
          const int pos = blk * 64 + (u & 3) * 16;
          if (blk >= p.nb) {
            atomicOr(p.status, BSA_DEV_BAD_INDEX);
          } else if (blk >= 0 && pos < len) {
            const int page = __ldg(table + blk);
            if (page < 0 || page >= p.num_pages) {
              atomicOr(p.status, BSA_DEV_BAD_INDEX);
            } else {
              my_n = min(16, len - pos);
              my_row = (page * p.Hkv + g) * 4 + (u & 3);
            }
          }
        }
        left = __ballot_sync(0xffffffffu, my_n > 0);
      }
      const int src = __ffs(left) - 1;
      left &= left - 1;
      row = __shfl_sync(0xffffffffu, my_row, src);
      n = __shfl_sync(0xffffffffu, my_n, src);
      return true;
    };
    uint4 kr[2][KH];          // rows r, r+8: 16 bytes of each half
    uint32_t vr[4][VW];       // rows 2c, 2c+1, 2c+8, 2c+9: D/8 bytes at r * D/8
    uint32_t ex = 0u;         // lane < 16: key exponent of row `lane`; else value exponent of row lane - 16
    auto load_k = [&]() {
      const uint8_t* k = p.k_pool + static_cast<int64_t>(row) * (16 * D);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int hf = 0; hf < KH; ++hf) kr[i][hf] = ld_stream(k + (r + 8 * i) * D + hf * 64 + c * 16);
      const uint8_t* e = lane < 16 ? p.k_exp : p.v_exp;
      ex = __ldg(e + static_cast<int64_t>(row) * 16 + (lane & 15));
    };
    auto load_v = [&]() {
      const uint8_t* v = p.v_pool + static_cast<int64_t>(row) * (16 * D);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* src = v + (2 * c + (i & 1) + 8 * (i >> 1)) * D + r * (D / 8);
        if constexpr (D == 128) {
          const uint4 t = ld_stream(src);
          vr[i][0] = t.x, vr[i][1] = t.y, vr[i][2] = t.z, vr[i][3] = t.w;
        } else {
          const uint2 t = __ldg(reinterpret_cast<const uint2*>(src));
          vr[i][0] = t.x, vr[i][1] = t.y;
        }
      }
    };

    bool more = next();
    if (more) {
      load_k();
      load_v();
    }
    while (more) {
      const int cur_n = n;
      // ---- S = K q^T: rows r, r+8 x heads 2c, 2c+1
      float S[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int hf = 0; hf < KH; ++hf) {
        const uint32_t a[4] = {kr[0][hf].x, kr[0][hf].y, kr[0][hf].z, kr[0][hf].w};
        const uint32_t e[4] = {kr[1][hf].x, kr[1][hf].y, kr[1][hf].z, kr[1][hf].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mma16816(S, cvt_e4m3x2(a[i]), cvt_e4m3x2(e[i]), cvt_e4m3x2(a[i] >> 16), cvt_e4m3x2(e[i] >> 16),
                   qf[hf * 4 + i][0], qf[hf * 4 + i][1]);
      }
      const uint32_t cur_ex = ex;
      more = next();
      if (more) load_k();
      // ---- weights
      float wgt[4];
      {
        float y[4], back[2];
        bool high = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int key = r + 8 * i;
          const bool in = key < cur_n;
          uint32_t ka = __shfl_sync(0xffffffffu, cur_ex, key);
          uint32_t va = __shfl_sync(0xffffffffu, cur_ex, 16 + key);
          if (!in) ka = va = 127u;
          const float kf = __uint_as_float(ka << 23);
          const float vb = static_cast<float>(static_cast<int>(va) - 127);
          back[i] = __uint_as_float((254u - va) << 23);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float v = S[2 * i + h] * kf * qs[h] + vb;
            y[2 * i + h] = in ? v : -INFINITY;
            high |= y[2 * i + h] > M[h] + kHeadroom;
          }
        }
        if (__any_sync(0xffffffffu, high)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float t = fmaxf(y[h], y[2 + h]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
            const float m_new = fmaxf(M[h], t);
            const float a = (m_new == -INFINITY) ? 1.0f : fast_exp2(M[h] - m_new);
            M[h] = m_new;
            l[h] *= a;
#pragma unroll
            for (int m = 0; m < MB; ++m) {
              O[m][h] *= a;
              O[m][2 + h] *= a;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float ref = (M[h] == -INFINITY) ? 0.0f : kLift - M[h];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            wgt[2 * i + h] = fast_exp2(y[2 * i + h] + ref);
            l[h] += wgt[2 * i + h] * back[i];
          }
        }
      }
      // keys x heads -> heads x keys: the B operand of O^T = V^T w
      const uint32_t b0 = transpose8x8(pack_f16x2(wgt[0], wgt[1]));
      const uint32_t b1 = transpose8x8(pack_f16x2(wgt[2], wgt[3]));
      if (cur_n < 16) {   // rows past the sequence may hold anything: a zero weight does not silence a NaN
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (2 * c + (i & 1) + 8 * (i >> 1) >= cur_n)
#pragma unroll
            for (int k = 0; k < VW; ++k) vr[i][k] = 0u;
      }
#pragma unroll
      for (int k = 0; k < VW; ++k) {
        // bytes of two keys side by side: channels (0,1) and (2,3) of this word
        const uint32_t lo01 = __byte_perm(vr[0][k], vr[1][k], 0x5140), lo23 = __byte_perm(vr[0][k], vr[1][k], 0x7362);
        const uint32_t hi01 = __byte_perm(vr[2][k], vr[3][k], 0x5140), hi23 = __byte_perm(vr[2][k], vr[3][k], 0x7362);
        mma16816(O[2 * k], cvt_e4m3x2(lo01), cvt_e4m3x2(lo01 >> 16), cvt_e4m3x2(hi01), cvt_e4m3x2(hi01 >> 16), b0, b1);
        mma16816(O[2 * k + 1], cvt_e4m3x2(lo23), cvt_e4m3x2(lo23 >> 16), cvt_e4m3x2(hi23), cvt_e4m3x2(hi23 >> 16), b0,
                 b1);
      }
      if (more) load_v();
    }

    // ---- join the warps of each set, then write the row or its partial record
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
    if (r == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // a NaN logit leaves M as it is; without another key the row must still not pass for an empty one
        if (M[h] == -INFINITY && l[h] != l[h]) M[h] = 0.0f;
        sh.m[warp][2 * c + h] = M[h];
        sh.l[warp][2 * c + h] = l[h];
      }
    }
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(&sh.o[warp][2 * c + h][pair_at<D>(r, m)]) = make_float2(O[m][h], O[m][2 + h]);
    __syncthreads();
    const bool whole = t0 == 0 && t1 == w;
    const int slot = t0 > 0 ? 0 : 1;
    for (int e = threadIdx.x; e < G * (D / 2); e += kThreads) {
      const int h = e / (D / 2), pr = e - h * (D / 2);         // query head of the group, channel pair
      const int hs = h >> 3, hh = h & 7;
      const int at = pair_at<D>(pr / (D / 16), pr % (D / 16));
      float mx = -INFINITY;
      for (int k = 0; k < per_set; ++k) mx = fmaxf(mx, sh.m[hs * per_set + k][hh]);
      float L = 0.0f, o0 = 0.0f, o1 = 0.0f;
      for (int k = 0; k < per_set; ++k) {
        const int wk = hs * per_set + k;
        const float mk = sh.m[wk][hh];
        if (mk == -INFINITY) continue;
        const float f = exp2f(mk - mx);
        const float2 v = *reinterpret_cast<const float2*>(&sh.o[wk][hh][at]);
        L += f * sh.l[wk][hh];
        o0 += f * v.x;
        o1 += f * v.y;
      }
      const int64_t orow = static_cast<int64_t>(b) * p.Hq + g * G + h;
      if (whole) {
        const float inv = (mx == -INFINITY) ? 0.0f : 1.0f / L;
        reinterpret_cast<uint32_t*>(p.o + orow * D)[pr] = pack_bf16x2(o0 * inv, o1 * inv);
        if (p.lse && pr == 0)
          p.lse[orow] = (mx == -INFINITY) ? -INFINITY : (mx - kLift + log2f(L)) * 0.69314718055994530942f;
      } else {
        float* rec = p.partial + ((static_cast<int64_t>(blockIdx.x) * 2 + slot) * G + h) * (D + 4);
        *reinterpret_cast<float2*>(rec + 4 + 2 * pr) = make_float2(o0, o1);
        if (pr == 0) {
          rec[0] = mx;
          rec[1] = L;
        }
      }
    }
    __syncthreads();
  }
}

// One block per (sequence, query head): rows cut by range borders are joined
// from their records, rows without a key become zero; rows that one range
// held are complete already.
template <int D>
__global__ void __launch_bounds__(D) combine_kernel(const QuantDecodeArgs p) {
  griddep_wait();
  __shared__ float red[D / 32], factor[D];
  const int G = p.Hq / p.Hkv;
  const int b = blockIdx.x / p.Hq, hq = blockIdx.x - b * p.Hq;
  const int g = hq / G, h = hq - g * G;
  const int tid = threadIdx.x;
  const int64_t orow = blockIdx.x;
  const int before = p.pre[b], w = p.pre[b + 1] - before;
  if (w == 0) {
    p.o[orow * D + tid] = __float2bfloat16_rn(0.0f);
    if (p.lse && tid == 0) p.lse[orow] = -INFINITY;
    return;
  }
  const int64_t total = static_cast<int64_t>(p.pre[p.B]) * p.Hkv;
  const int C = ranges(total, p.num_ctas);
  const int64_t x0 = static_cast<int64_t>(before) * p.Hkv + static_cast<int64_t>(g) * w;
  const int first = cta_of(x0, total, C), n = cta_of(x0 + w - 1, total, C) - first + 1;
  if (n == 1) return;
  // the row begins inside range `first` (its record 1) and goes on in the next ones (their records 0)
  const float* rec = p.partial + (static_cast<int64_t>(first) * 2 * G + h) * (D + 4);
  const int step = 2 * G * (D + 4);
  auto record = [&](int k) { return rec + (k == 0 ? G * (D + 4) : static_cast<int64_t>(k) * step); };
  float mx = -INFINITY;
  for (int k = tid; k < n; k += D) mx = fmaxf(mx, record(k)[0]);
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if ((tid & 31) == 0) red[tid >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < D / 32; ++k) mx = fmaxf(mx, red[k]);
  __syncthreads();
  // records D at a time: thread = record for their factors, then thread = channel
  float L = 0.0f, acc = 0.0f;
  for (int k0 = 0; k0 < n; k0 += D) {
    float f = 0.0f;
    if (k0 + tid < n && mx != -INFINITY) {
      const float2 ml = *reinterpret_cast<const float2*>(record(k0 + tid));
      f = exp2f(ml.x - mx);     // 0 where the record is empty
      L += f * ml.y;
    }
    factor[tid] = f;
    __syncthreads();
    const int m = min(D, n - k0);
#pragma unroll 8
    for (int k = 0; k < m; ++k) acc += factor[k] * record(k0 + k)[4 + tid];
    __syncthreads();
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if ((tid & 31) == 0) red[tid >> 5] = L;
  __syncthreads();
  L = 0.0f;
#pragma unroll
  for (int k = 0; k < D / 32; ++k) L += red[k];
  p.o[orow * D + tid] = __float2bfloat16_rn(mx == -INFINITY ? 0.0f : acc / L);
  if (p.lse && tid == 0) p.lse[orow] = (mx == -INFINITY) ? -INFINITY : (mx - kLift + log2f(L)) * 0.69314718055994530942f;
}

template <int D>
cudaError_t launch(const QuantDecodeArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(Shared<D>) + (static_cast<size_t>(a.B) + 1) * sizeof(int);
  cudaError_t e = ensure_dynamic_smem<decode_kernel<D>>(smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(decode_kernel<D>, dim3(a.num_ctas), dim3(kThreads), smem, st, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(combine_kernel<D>, dim3(a.B * a.Hq), dim3(D), 0, st, a);
}

}  // namespace qdecode

int quant_decode_ctas(int num_sms) { return qdecode::kCtasPerSm * num_sms; }

cudaError_t launch_attn_decode_quant(const QuantDecodeArgs& a, int d, cudaStream_t st) {
  return d == 64 ? qdecode::launch<64>(a, st) : qdecode::launch<128>(a, st);
}

}  // namespace bsa
