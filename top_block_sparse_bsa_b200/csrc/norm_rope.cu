// norm_rope.cu -- from a fused projection to the attention's inputs: the
// RMS norm of each query and key head, the rotation by the token's position,
// and the change from token-major to head-major, in one pass; and its
// backward.
//
// Formulas.  For a row x of d channels (one head of one token), weight w:
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r w
//   pair (a, b) of the first rot_dim channels, angle t = position * inv_freq:
//     (a, b) -> s (a cos t - b sin t, a sin t + b cos t)
// Backward, dz the gradient of the output row: dy = the rotation by -t of dz
// (times s), dw = sum over rows of dy x r, dx = r (dy w - x r^2 mean(dy w x)).
//
// Both passes are bound by memory: every value is read once and written once
// and a row needs about 10 operations a channel.  So a row lives in the
// registers of d/8 lanes (rounded up to 8, 16 or 32), eight channels a lane in
// two pieces of four.  In the half layout a lane's pieces are channels i..i+3
// and their partners rot_dim/2 further, so the rotation needs no exchange
// between lanes; the sums of the norm are shuffles inside the row's lanes.
// A lane keeps its channels from head to head, so the cosines and sines of a
// token are computed once per lane and serve all its heads: no table of
// angles is read.
//
// Angles.  position * inv_freq reaches 1e6 radians and more, where an fp32
// product is off by 0.06.  The frequency in turns, modulo one, is held as a
// 64-bit fixed-point fraction; the integer product with the position wraps
// modulo one turn exactly, and its top 32 bits are the angle to 2^-32 turns.
#include "common.cuh"
#include "kernels.h"

namespace bsa {
namespace nrope {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;   // rows a lane has in flight

enum { LAYOUT_NONE = 0, LAYOUT_HALF = 1, LAYOUT_PAIRS = 2 };

// Four consecutive channels of a row.
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 t = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 t = __ldg(reinterpret_cast<const uint2*>(p));
  v[0] = __uint_as_float(t.x << 16); v[1] = __uint_as_float(t.x & 0xFFFF0000u);
  v[2] = __uint_as_float(t.y << 16); v[3] = __uint_as_float(t.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
// The one rounding of the operator: fp32 results to the output's type.
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// The channels of one lane: pieces [a, a+4) and [b, b+4); `on`: they exist;
// `rotated`: they belong to the rotated part.  rot is a multiple of 8.
struct Lane {
  int a, b;
  bool on, rotated;
};
template <int LAYOUT>
__device__ __forceinline__ Lane lane_channels(int l, int d, int rot) {
  Lane m;
  if (LAYOUT == LAYOUT_HALF && l < rot / 8) {
    m.a = 4 * l;
    m.b = rot / 2 + 4 * l;
  } else {
    m.a = 8 * l;
    m.b = 8 * l + 4;
  }
  m.on = 8 * l < d;
  m.rotated = LAYOUT != LAYOUT_NONE && 8 * l < rot;
  return m;
}

// The lane's four frequencies as fractions of a turn, 2^64 to the turn.
__device__ __forceinline__ void lane_freqs(const double* __restrict__ inv_freq, int l, bool rotated,
                                           unsigned long long (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = 0;
    if (rotated) {
      double t = __ldg(inv_freq + 4 * l + i) * 0.15915494309189533577;   // 1 / (2 pi)
      t -= floor(t);
      f[i] = __double2ull_rd(t * 18446744073709551616.0);
    }
  }
}
__device__ __forceinline__ void angles(const unsigned long long (&f)[4], int pos, float scale, float (&c)[4],
                                       float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned long long turns = static_cast<unsigned long long>(static_cast<long long>(pos)) * f[i];
    const int top = static_cast<int>(turns >> 32);
    float sn, cs;
    sincospif(static_cast<float>(top) * 4.656612873077392578125e-10f, &sn, &cs);   // half turns: 2^-31
    c[i] = cs * scale;
    s[i] = sn * scale;
  }
}
// (a, b) turned by (c, s); the half layout pairs a[i] with b[i], the other one
// neighbours inside each piece.
template <int LAYOUT>
__device__ __forceinline__ void rotate(float (&a)[4], float (&b)[4], const float (&c)[4], const float (&s)[4]) {
  if (LAYOUT == LAYOUT_HALF) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[i], y = b[i];
      a[i] = x * c[i] - y * s[i];
      b[i] = x * s[i] + y * c[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x = a[2 * i], y = a[2 * i + 1];
      a[2 * i] = x * c[i] - y * s[i];
      a[2 * i + 1] = x * s[i] + y * c[i];
      x = b[2 * i], y = b[2 * i + 1];
      b[2 * i] = x * c[2 + i] - y * s[2 + i];
      b[2 * i + 1] = x * s[2 + i] + y * c[2 + i];
    }
  }
}

template <int GS>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = GS / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Work items: token tiles (kThreads/GS tokens, one per lane group) x runs of
// head_run heads.
template <typename T, int GS, int LAYOUT>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const NormRopeArgs p) {
  griddep_wait();
  constexpr int kTokens = kThreads / GS;
  const int l = threadIdx.x % GS, grp = threadIdx.x / GS;
  const Lane m = lane_channels<LAYOUT>(l, p.d, p.rot);
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kTokens + grp;
  const int64_t tokens = static_cast<int64_t>(p.B) * p.N;
  const bool live = token < tokens;      // lanes of a dead group still take part in the shuffles
  const int64_t tk = live ? token : 0;
  const int b = static_cast<int>(tk / p.N);
  const int n = static_cast<int>(tk - static_cast<int64_t>(b) * p.N);
  const int h_begin = blockIdx.y * p.head_run, h_end = min(h_begin + p.head_run, p.Hq + 2 * p.Hkv);
  const T* row0 = static_cast<const T*>(p.qkv) + tk * p.token_stride;
  float c[4], s[4];
  if (LAYOUT != LAYOUT_NONE && h_begin < p.Hq + p.Hkv) {
    unsigned long long f[4];
    lane_freqs(p.inv_freq, l, m.rotated, f);
    angles(f, p.positions ? __ldg(p.positions + tk) : n, p.rope_scale, c, s);
  }
  for (int part = 0; part < 3; ++part) {   // queries, keys, values
    const int lo = part == 0 ? 0 : (part == 1 ? p.Hq : p.Hq + p.Hkv);
    const int heads = part == 0 ? p.Hq : p.Hkv;
    const int from = max(h_begin, lo), to = min(h_end, lo + heads);
    if (from >= to) continue;
    const T* weight = static_cast<const T*>(part == 0 ? p.q_weight : p.k_weight);
    T* out = static_cast<T*>(part == 0 ? p.q : (part == 1 ? p.k : p.v));
    const bool norm = part < 2 && weight != nullptr;
    float wa[4], wb[4];
    if (norm && m.on) {
      load4(weight + m.a, wa);
      load4(weight + m.b, wb);
    }
    for (int h0 = from; h0 < to; h0 += kUnroll) {
      float xa[kUnroll][4], xb[kUnroll][4];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (m.on && live && h0 + u < to) {
          load4(row0 + static_cast<int64_t>(h0 + u) * p.d + m.a, xa[u]);
          load4(row0 + static_cast<int64_t>(h0 + u) * p.d + m.b, xb[u]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) xa[u][i] = xb[u][i] = 0.0f;
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (norm) {
          float ss = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) ss += xa[u][i] * xa[u][i] + xb[u][i] * xb[u][i];
          const float r = rsqrtf(row_sum<GS>(ss) * p.inv_d + p.eps);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            xa[u][i] *= r * wa[i];
            xb[u][i] *= r * wb[i];
          }
        }
        if (LAYOUT != LAYOUT_NONE && part < 2 && m.rotated) rotate<LAYOUT>(xa[u], xb[u], c, s);
        if (m.on && live && h0 + u < to) {
          T* dst = out + ((static_cast<int64_t>(b) * heads + (h0 + u - lo)) * p.N + n) * p.d;
          store4(dst + m.a, xa[u]);
          store4(dst + m.b, xb[u]);
        }
      }
    }
  }
}

// Backward.  Persistent over (token tile, head run) items; each lane sums the
// weights' gradients of its channels over all its rows in fp32, the block's
// groups are added in order at the end, and dw_reduce_kernel adds the blocks
// in 64 bits: the same order on every run.
template <typename T, int GS, int LAYOUT>
__global__ void __launch_bounds__(kThreads) bwd_kernel(const NormRopeArgs p) {
  griddep_wait();
  constexpr int kTokens = kThreads / GS;
  constexpr int kRows = 2;   // rows a lane has in flight (their fp32 gradients and inputs)
  __shared__ float acc[2][kTokens][GS * 8];
  const int l = threadIdx.x % GS, grp = threadIdx.x / GS;
  const Lane m = lane_channels<LAYOUT>(l, p.d, p.rot);
  const int64_t tokens = static_cast<int64_t>(p.B) * p.N;
  const int64_t tiles = (tokens + kTokens - 1) / kTokens;
  const int H = p.Hq + 2 * p.Hkv;
  const int runs = (H + p.head_run - 1) / p.head_run;
  const bool norm = p.q_weight != nullptr;
  unsigned long long f[4];
  if (LAYOUT != LAYOUT_NONE) lane_freqs(p.inv_freq, l, m.rotated, f);
  float dwa[2][4] = {}, dwb[2][4] = {};
  for (int64_t item = blockIdx.x; item < tiles * runs; item += gridDim.x) {
    const int64_t tile = item / runs;
    const int run = static_cast<int>(item - tile * runs);
    const int64_t token = tile * kTokens + grp;
    const bool live = token < tokens;
    const int64_t tk = live ? token : 0;
    const int b = static_cast<int>(tk / p.N);
    const int n = static_cast<int>(tk - static_cast<int64_t>(b) * p.N);
    const int h_begin = run * p.head_run, h_end = min(h_begin + p.head_run, H);
    const T* row0 = static_cast<const T*>(p.qkv) + tk * p.token_stride;
    T* drow0 = static_cast<T*>(p.d_qkv) + tk * p.d_token_stride;
    float c[4], s[4];
    if (LAYOUT != LAYOUT_NONE && h_begin < p.Hq + p.Hkv) {
      angles(f, p.positions ? __ldg(p.positions + tk) : n, p.rope_scale, c, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = -s[i];
    }
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      const int lo = part == 0 ? 0 : (part == 1 ? p.Hq : p.Hq + p.Hkv);
      const int heads = part == 0 ? p.Hq : p.Hkv;
      const int from = max(h_begin, lo), to = min(h_end, lo + heads);
      if (from >= to) continue;
      const float* dz = part == 0 ? p.dq : (part == 1 ? p.dk : p.dv);
      const T* weight = static_cast<const T*>(part == 0 ? p.q_weight : p.k_weight);
      const bool nm = part < 2 && norm;
      float wa[4], wb[4];
      if (nm && m.on) {
        load4(weight + m.a, wa);
        load4(weight + m.b, wb);
      }
      for (int h0 = from; h0 < to; h0 += kRows) {
        float ga[kRows][4], gb[kRows][4], xa[kRows][4], xb[kRows][4];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const bool in = m.on && live && h0 + u < to;
#pragma unroll
          for (int i = 0; i < 4; ++i) ga[u][i] = gb[u][i] = xa[u][i] = xb[u][i] = 0.0f;
          if (in) {
            const float* src = dz + ((static_cast<int64_t>(b) * heads + (h0 + u - lo)) * p.N + n) * p.d;
            load4(src + m.a, ga[u]);
            load4(src + m.b, gb[u]);
            if (nm) {
              load4(row0 + static_cast<int64_t>(h0 + u) * p.d + m.a, xa[u]);
              load4(row0 + static_cast<int64_t>(h0 + u) * p.d + m.b, xb[u]);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          if (LAYOUT != LAYOUT_NONE && part < 2 && m.rotated) rotate<LAYOUT>(ga[u], gb[u], c, s);
          if (nm) {
            float ss = 0.0f, sd = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              ss += xa[u][i] * xa[u][i] + xb[u][i] * xb[u][i];
              if (m.on) sd += ga[u][i] * wa[i] * xa[u][i] + gb[u][i] * wb[i] * xb[u][i];
            }
            ss = row_sum<GS>(ss);
            sd = row_sum<GS>(sd);
            const float r = rsqrtf(ss * p.inv_d + p.eps);
            const float k = r * r * sd * p.inv_d;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (m.on) {
                dwa[part & 1][i] += ga[u][i] * xa[u][i] * r;
                dwb[part & 1][i] += gb[u][i] * xb[u][i] * r;
                ga[u][i] = r * (ga[u][i] * wa[i] - xa[u][i] * k);
                gb[u][i] = r * (gb[u][i] * wb[i] - xb[u][i] * k);
              }
            }
          }
          if (m.on && live && h0 + u < to) {
            T* dst = drow0 + static_cast<int64_t>(h0 + u) * p.d;
            store4(dst + m.a, ga[u]);
            store4(dst + m.b, gb[u]);
          }
        }
      }
    }
  }
  if (!norm) return;
  if (m.on) {
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[w][grp][m.a + i] = dwa[w][i];
        acc[w][grp][m.b + i] = dwb[w][i];
      }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * p.d; e += kThreads) {
    const int w = e / p.d, ch = e - w * p.d;
    float v = 0.0f;
#pragma unroll
    for (int g = 0; g < kTokens; ++g) v += acc[w][g][ch];
    p.dw_partial[static_cast<int64_t>(blockIdx.x) * 2 * p.d + e] = v;
  }
}

// dw[e] = the blocks' partial sums, e over both weights' channels: 32 outputs
// a block, eight threads each, added in 64 bits in a fixed order.
__global__ void __launch_bounds__(256) dw_reduce_kernel(const float* __restrict__ partial, int blocks, int d,
                                                        float* __restrict__ dqw, float* __restrict__ dkw) {
  griddep_wait();
  __shared__ double part[8][32];
  const int col = threadIdx.x % 32, row = threadIdx.x / 32;
  const int e = blockIdx.x * 32 + col;
  double v = 0.0;
  if (e < 2 * d)
    for (int k = row; k < blocks; k += 8) v += static_cast<double>(partial[static_cast<int64_t>(k) * 2 * d + e]);
  part[row][col] = v;
  __syncthreads();
  if (row == 0 && e < 2 * d) {
#pragma unroll
    for (int k = 1; k < 8; ++k) v += part[k][col];
    (e < d ? dqw[e] : dkw[e - d]) = static_cast<float>(v);
  }
}

template <typename T, int GS, int LAYOUT>
cudaError_t launch(NormRopeArgs p, bool bwd, int num_sms, cudaStream_t st) {
  constexpr int kTokens = kThreads / GS;
  const int64_t tiles = (static_cast<int64_t>(p.B) * p.N + kTokens - 1) / kTokens;
  const int H = p.Hq + 2 * p.Hkv;
  // heads of one token are split over blocks only while the token tiles alone
  // leave multiprocessors without two blocks
  int runs = 1;
  while (runs < H && tiles * runs < 2 * num_sms) runs *= 2;
  p.head_run = (H + runs - 1) / runs;
  runs = (H + p.head_run - 1) / p.head_run;
  if (!bwd)
    return launch_dependent(fwd_kernel<T, GS, LAYOUT>, dim3(static_cast<unsigned>(tiles), runs), dim3(kThreads), 0, st,
                            p);
  const int64_t items = tiles * runs;
  const int grid = static_cast<int>(items < norm_rope_bwd_blocks(num_sms) ? items : norm_rope_bwd_blocks(num_sms));
  cudaError_t e = launch_dependent(bwd_kernel<T, GS, LAYOUT>, dim3(grid), dim3(kThreads), 0, st, p);
  if (e != cudaSuccess || p.q_weight == nullptr) return e;
  return launch_dependent(dw_reduce_kernel, dim3((2 * p.d + 31) / 32), dim3(256), 0, st, p.dw_partial, grid, p.d,
                          p.d_q_weight, p.d_k_weight);
}

template <typename T, int GS>
cudaError_t by_layout(const NormRopeArgs& p, bool bwd, int num_sms, cudaStream_t st) {
  if (p.layout == LAYOUT_HALF) return launch<T, GS, LAYOUT_HALF>(p, bwd, num_sms, st);
  if (p.layout == LAYOUT_PAIRS) return launch<T, GS, LAYOUT_PAIRS>(p, bwd, num_sms, st);
  return launch<T, GS, LAYOUT_NONE>(p, bwd, num_sms, st);
}
template <typename T>
cudaError_t by_width(const NormRopeArgs& p, bool bwd, int num_sms, cudaStream_t st) {
  if (p.d <= 64) return by_layout<T, 8>(p, bwd, num_sms, st);
  if (p.d <= 128) return by_layout<T, 16>(p, bwd, num_sms, st);
  return by_layout<T, 32>(p, bwd, num_sms, st);
}

}  // namespace nrope

int norm_rope_bwd_blocks(int num_sms) { return 4 * num_sms; }

cudaError_t launch_norm_rope(const NormRopeArgs& a, bool bf16, bool bwd, int num_sms, cudaStream_t st) {
  return bf16 ? nrope::by_width<__nv_bfloat16>(a, bwd, num_sms, st) : nrope::by_width<float>(a, bwd, num_sms, st);
}

}  // namespace bsa
