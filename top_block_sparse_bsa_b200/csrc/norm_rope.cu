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
// registers of a few lanes, 2 E channels a lane in two pieces of E = 4 or 8.  In
// the half layout a lane's pieces are channels i..i+E-1 and their partners
// rot_dim/2 further, so the rotation needs no exchange between lanes; the sums
// of the norm are shuffles inside the row's lanes.  A lane keeps its channels
// from head to head, so the cosines and sines of a token are computed once per
// lane and serve all its heads: no table of angles is read.  32K tokens of 48
// heads, bf16: 134 to 137 us, 89 to 91% of the copy rate; fp32 254 us, 97%; the
// backward of 32K tokens of 36 heads 204 to 218 us (82 to 88%, by box and
// clock), with fp32 inputs 273 us, 97%.
//
// Angles.  position * inv_freq reaches 1e6 radians and more, where an fp32
// product is off by 0.06.  The frequency in turns, modulo one, is held as a
// 64-bit fixed-point fraction; the integer product with the position wraps
// modulo one turn exactly.  What is left: the top 32 bits become an fp32 argument
// (2^-26 turns), and the frequency's own rounding in 64 bits, 2^-55 turns for
// frequencies up to 1, grows with the position (2^-24 turns at the ends of int32).
#include "common.cuh"
#include "kernels.h"

namespace bsa {
namespace nrope {

constexpr int kThreads = 256;
// Rows a lane of the forward has in flight, and blocks an SM (32K tokens of 48
// heads, us): bf16 in 16-byte pieces 4 rows x 2 blocks 135, 3 x 2 147, 5 x 2 143,
// 6 x 2 150, 2 x 3 154; in 8-byte pieces 4 x 4 143, 3 x 4 147, 2 x 5 145; fp32
// 3 x 3 252, 4 x 3 257, 4 x 4 280.
template <typename T, int E>
__host__ __device__ constexpr int fwd_rows() {
  return sizeof(T) == 4 ? 3 : 4;
}
template <typename T, int E>
__host__ __device__ constexpr int fwd_ctas() {
  return sizeof(T) == 4 ? 3 : (E == 8 ? 2 : 4);
}
constexpr int kBwdCtasPerSm = 2;
template <typename T>
__host__ __device__ constexpr int bwd_rows() {
  return sizeof(T) == 2 ? 4 : 2;
}

enum { LAYOUT_NONE = 0, LAYOUT_HALF = 1, LAYOUT_PAIRS = 2 };

// E consecutive channels of a row, kept as loaded: a bf16 piece waits for its
// turn in half of the registers.  pairs() gives them as packed fp32 pairs.
template <typename T, int E>
struct Raw;
template <>
struct Raw<float, 4> {
  float4 v;
  __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void fill(uint32_t bits) {
    v.x = v.y = v.z = v.w = __uint_as_float(bits);
  }
  __device__ __forceinline__ void load(const float* p) { v = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
  __device__ __forceinline__ void pairs(uint64_t* x) const {
    x[0] = f2_pack(v.x, v.y);
    x[1] = f2_pack(v.z, v.w);
  }
};
__device__ __forceinline__ uint64_t widen(uint32_t two) {
  return f2_pack(__uint_as_float(two << 16), __uint_as_float(two & 0xFFFF0000u));
}
template <>
struct Raw<__nv_bfloat16, 4> {
  uint2 v;
  __device__ __forceinline__ void zero() { v = make_uint2(0u, 0u); }
  __device__ __forceinline__ void fill(uint32_t bits) { v = make_uint2(bits, bits); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = v; }
  __device__ __forceinline__ void pairs(uint64_t* x) const {
    x[0] = widen(v.x);
    x[1] = widen(v.y);
  }
};
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void pairs(uint64_t* x) const {
    x[0] = widen(v.x);
    x[1] = widen(v.y);
    x[2] = widen(v.z);
    x[3] = widen(v.w);
  }
};
// The one rounding of the operator: fp32 results to the output's type.
__device__ __forceinline__ uint32_t narrow(uint64_t x) {
  float lo, hi;
  f2_unpack(x, lo, hi);
  return pack_bf16x2(lo, hi);
}
template <typename T, int E>
__device__ __forceinline__ void store_pairs(T* p, const uint64_t* x) {
  if constexpr (sizeof(T) == 4) {
    float4 v;
    f2_unpack(x[0], v.x, v.y);
    f2_unpack(x[1], v.z, v.w);
    *reinterpret_cast<float4*>(p) = v;
  } else if constexpr (E == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(narrow(x[0]), narrow(x[1]));
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(narrow(x[0]), narrow(x[1]), narrow(x[2]), narrow(x[3]));
  }
}

// The channels of one lane: pieces [a, a+E) and [b, b+E); `on`: they exist;
// `rotated`: they belong to the rotated part.  d and rot are multiples of 2 E.
struct Lane {
  int a, b;
  bool on, rotated;
};
template <int LAYOUT, int E>
__device__ __forceinline__ Lane lane_channels(int l, int d, int rot) {
  Lane m;
  if (LAYOUT == LAYOUT_HALF && 2 * E * l < rot) {
    m.a = E * l;
    m.b = rot / 2 + E * l;
  } else {
    m.a = 2 * E * l;
    m.b = 2 * E * l + E;
  }
  m.on = 2 * E * l < d;
  m.rotated = LAYOUT != LAYOUT_NONE && 2 * E * l < rot;
  return m;
}

template <typename T, int E>
__device__ __forceinline__ void load_weight(const T* __restrict__ weight, const Lane& m, float (&w)[2 * E]) {
  Raw<T, E> a, b;
  a.load(weight + m.a);
  b.load(weight + m.b);
  uint64_t x[E];
  a.pairs(x);
  b.pairs(x + E / 2);
#pragma unroll
  for (int k = 0; k < E; ++k) f2_unpack(x[k], w[2 * k], w[2 * k + 1]);
}

// Frequencies as fractions of a turn, 2^64 to the turn, in shared memory: one
// conversion a block and pair.  A lane's E begin at E l.
constexpr int kMaxPairs = 128;
__device__ __forceinline__ void block_freqs(const double* __restrict__ inv_freq, int pairs,
                                            unsigned long long* __restrict__ f) {
  for (int i = threadIdx.x; i < pairs; i += kThreads) {
    double t = __ldg(inv_freq + i) * 0.15915494309189533577;   // 1 / (2 pi)
    t -= floor(t);
    f[i] = __double2ull_rd(t * 18446744073709551616.0);
  }
  __syncthreads();
}
template <int E>
__device__ __forceinline__ void angles(const unsigned long long* __restrict__ f, int pos, float scale, float (&c)[E],
                                       float (&s)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const unsigned long long turns = static_cast<unsigned long long>(static_cast<long long>(pos)) * f[i];
    const int top = static_cast<int>(turns >> 32);
    float sn, cs;
    sincospif(static_cast<float>(top) * 4.656612873077392578125e-10f, &sn, &cs);   // half turns: 2^-31
    c[i] = cs * scale;
    s[i] = sn * scale;
  }
}
// A lane's 2 E channels as packed pairs X[0..E-1], piece a's (a0,a1) (a2,a3) ...
// and then b's.  A rotation (with factors on the channels) is P X + Q X', where
// X' is the pair that holds X's partners: X[k ^ E/2] in the half layout, X
// itself with its two halves exchanged in the other.
template <int LAYOUT, int E>
__device__ __forceinline__ uint64_t partner(const uint64_t (&x)[E], int k) {
  if (LAYOUT == LAYOUT_HALF) return x[k ^ (E / 2)];
  float lo, hi;
  f2_unpack(x[k], lo, hi);
  return f2_pack(hi, lo);
}
// P and Q of the turn by (c, s) of channels whose factors are w: y = turn(w x).
template <int LAYOUT, int E>
__device__ __forceinline__ void turn_factors(const float (&c)[E], const float (&s)[E], const float (&w)[2 * E],
                                             uint64_t (&P)[E], uint64_t (&Q)[E]) {
#pragma unroll
  for (int k = 0; k < E; ++k) {
    const int i0 = 2 * k, i1 = 2 * k + 1;              // the pair's channels among the lane's
    if (LAYOUT == LAYOUT_HALF) {
      const int q = i0 & (E - 1), o = i0 ^ E;          // angles of the pair; partners o, o + 1
      const float sign = k < E / 2 ? -1.0f : 1.0f;
      P[k] = f2_pack(w[i0] * c[q], w[i1] * c[q + 1]);
      Q[k] = f2_pack(sign * w[o] * s[q], sign * w[o + 1] * s[q + 1]);
    } else {
      P[k] = f2_pack(w[i0] * c[k], w[i1] * c[k]);
      Q[k] = f2_pack(-w[i1] * s[k], w[i0] * s[k]);
    }
  }
}

template <int GS>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = GS / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Forward: one block per token tile (kThreads / GS tokens, one per lane group)
// and run of head_run heads.  Blocks that start as others end do better here
// than resident ones with even shares (144 us against 181 for 32K tokens, both in
// 8-byte pieces: these run in step, all loading or all storing, and the split
// costs registers).
template <typename T, int GS, int LAYOUT, int E>
__global__ void __launch_bounds__(kThreads, fwd_ctas<T, E>()) fwd_kernel(const NormRopeArgs p) {
  griddep_wait();
  constexpr int kTokens = kThreads / GS, kUnroll = fwd_rows<T, E>();
  __shared__ unsigned long long freqs[kMaxPairs];
  const int l = threadIdx.x % GS, grp = threadIdx.x / GS;
  const Lane m = lane_channels<LAYOUT, E>(l, p.d, p.rot);
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kTokens + grp;
  const int64_t tokens = static_cast<int64_t>(p.B) * p.N;
  const bool live = token < tokens;      // lanes of a dead group still take part in the shuffles
  const int64_t tk = live ? token : 0;
  const int b = static_cast<int>(tk / p.N);
  const int n = static_cast<int>(tk - static_cast<int64_t>(b) * p.N);
  const int h_begin = blockIdx.y * p.head_run, h_end = min(h_begin + p.head_run, p.Hq + 2 * p.Hkv);
  const T* row0 = static_cast<const T*>(p.qkv) + tk * p.token_stride;
  float c[E], s[E];
  if (LAYOUT != LAYOUT_NONE && h_begin < p.Hq + p.Hkv) {
    block_freqs(p.inv_freq, p.rot / 2, freqs);
    if (m.rotated) angles<E>(freqs + E * l, p.positions ? __ldg(p.positions + tk) : n, p.rope_scale, c, s);
  }
  for (int part = 0; part < 3; ++part) {   // queries, keys, values
    const int lo = part == 0 ? 0 : (part == 1 ? p.Hq : p.Hq + p.Hkv);
    const int heads = part == 0 ? p.Hq : p.Hkv;
    const int from = max(h_begin, lo), to = min(h_end, lo + heads);
    if (from >= to) continue;
    const T* weight = static_cast<const T*>(part == 0 ? p.q_weight : p.k_weight);
    const T* src = row0 + from * p.d;
    const int64_t head_step = static_cast<int64_t>(p.N) * p.d;
    T* dst = static_cast<T*>(part == 0 ? p.q : (part == 1 ? p.k : p.v)) +
             (static_cast<int64_t>(b) * heads + (from - lo)) * head_step + static_cast<int64_t>(n) * p.d;
    const bool norm = part < 2 && weight != nullptr;
    const bool turned = LAYOUT != LAYOUT_NONE && part < 2 && m.rotated;
    // the norm's weight rides in the rotation's factors; without a rotation P is the weight alone
    uint64_t P[E], Q[E];
    if (part < 2) {
      float w[2 * E];
#pragma unroll
      for (int i = 0; i < 2 * E; ++i) w[i] = 1.0f;
      if (norm && m.on) load_weight<T, E>(weight, m, w);
      if (turned) {
        turn_factors<LAYOUT, E>(c, s, w, P, Q);
      } else {
#pragma unroll
        for (int k = 0; k < E; ++k) P[k] = f2_pack(w[2 * k], w[2 * k + 1]), Q[k] = 0;
      }
    }
    for (int h0 = from; h0 < to; h0 += kUnroll, src += kUnroll * p.d, dst += kUnroll * head_step) {
      Raw<T, E> ra[kUnroll], rb[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (m.on && live && h0 + u < to) {
          ra[u].load(src + u * p.d + m.a);
          rb[u].load(src + u * p.d + m.b);
        } else {
          ra[u].zero();
          rb[u].zero();
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const bool in = m.on && live && h0 + u < to;
        T* to_row = dst + u * head_step;
        if (part == 2) {
          if (in) {
            ra[u].store(to_row + m.a);
            rb[u].store(to_row + m.b);
          }
          continue;
        }
        uint64_t x[E], y[E];
        ra[u].pairs(x);
        rb[u].pairs(x + E / 2);
#pragma unroll
        for (int k = 0; k < E; ++k) y[k] = f2_mul(P[k], x[k]);
        if (turned) {
#pragma unroll
          for (int k = 0; k < E; ++k) y[k] = f2_fma(Q[k], partner<LAYOUT, E>(x, k), y[k]);
        }
        if (norm) {
          uint64_t s2 = f2_mul(x[0], x[0]);
#pragma unroll
          for (int k = 1; k < E; ++k) s2 = f2_fma(x[k], x[k], s2);
          float lo2, hi2;
          f2_unpack(s2, lo2, hi2);
          const float r = rsqrtf(row_sum<GS>(lo2 + hi2) * p.inv_d + p.eps);
          const uint64_t rr = f2_pack(r, r);
#pragma unroll
          for (int k = 0; k < E; ++k) y[k] = f2_mul(y[k], rr);
        }
        if (in) {
          store_pairs<T, E>(to_row + m.a, y);
          store_pairs<T, E>(to_row + m.b, y + E / 2);
        }
      }
    }
  }
}

// Work split of the backward: token tiles x heads, laid end to end tile by tile
// in units of head_run heads and cut into one even range a block, all blocks
// resident at once; a block forms a token's angles once for each stretch of its
// heads.
struct Stretch {
  int64_t tile;
  int h_begin, h_end;
};
struct Range {
  int64_t x, hi;
  int units, run, H;
  __device__ __forceinline__ Range(const NormRopeArgs& p, int tile_tokens) {
    H = p.Hq + 2 * p.Hkv;
    run = p.head_run;
    units = (H + run - 1) / run;
    const int64_t tiles = (static_cast<int64_t>(p.B) * p.N + tile_tokens - 1) / tile_tokens;
    x = blockIdx.x * (tiles * units) / gridDim.x;
    hi = (blockIdx.x + 1) * (tiles * units) / gridDim.x;
  }
  __device__ __forceinline__ bool next(Stretch& t) {
    if (x >= hi) return false;
    t.tile = x / units;
    const int u0 = static_cast<int>(x - t.tile * units);
    const int u1 = static_cast<int>(min(static_cast<int64_t>(units), u0 + (hi - x)));
    t.h_begin = u0 * run;
    t.h_end = min(u1 * run, H);
    x += u1 - u0;
    return true;
  }
};

// Backward.  The weights'
// gradients of a lane's channels are summed in registers over the heads of a
// token and added to the lane's own place in shared memory token by token
// (which frees half of the registers that sums over all rows would hold); the
// block's groups are added in order at the end, and dw_reduce_kernel adds the
// blocks in 64 bits: the same order on every run.  Inside a block the sums are
// fp32: a block sees 1/296 of the rows, and sums in 64 bits would take twice the
// registers and shared memory of the part that bounds the pass.
template <typename T, int GS, int LAYOUT>
__global__ void __launch_bounds__(kThreads, kBwdCtasPerSm) bwd_kernel(const NormRopeArgs p) {
  griddep_wait();
  constexpr int kTokens = kThreads / GS;
  constexpr int kRows = bwd_rows<T>();   // rows a lane has in flight (their fp32 gradients and inputs)
  __shared__ float4 acc[2][2][kThreads];   // [weight][piece][thread]
  __shared__ unsigned long long freqs[kMaxPairs];
  const int l = threadIdx.x % GS, grp = threadIdx.x / GS;
  const Lane m = lane_channels<LAYOUT, 4>(l, p.d, p.rot);
  const bool norm = p.q_weight != nullptr;
  // rows past the last head: ones, with gradients of zero.  Zeros would have an infinite 1/rms where eps is 0, and
  // 0 times that is a NaN in the weights' sums.
  const uint32_t pad = !m.on ? 0u : (sizeof(T) == 2 ? 0x3F803F80u : 0x3F800000u);
  if (LAYOUT != LAYOUT_NONE) block_freqs(p.inv_freq, p.rot / 2, freqs);
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i >> 1][i & 1][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  Range work(p, kTokens);
  for (Stretch st; work.next(st);) {
    const int64_t token = st.tile * kTokens + grp;
    const bool live = token < static_cast<int64_t>(p.B) * p.N;
    const int64_t tk = live ? token : 0;
    const int b = static_cast<int>(tk / p.N);
    const int n = static_cast<int>(tk - static_cast<int64_t>(b) * p.N);
    const int h_begin = st.h_begin, h_end = st.h_end;
    const T* row0 = static_cast<const T*>(p.qkv) + tk * p.token_stride;
    T* drow0 = static_cast<T*>(p.d_qkv) + tk * p.d_token_stride;
    uint64_t P[4] = {}, Q[4] = {};
    if (LAYOUT != LAYOUT_NONE && m.rotated && h_begin < p.Hq + p.Hkv) {
      float c[4], s[4];
      angles<4>(freqs + 4 * l, p.positions ? __ldg(p.positions + tk) : n, p.rope_scale, c, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = -s[i];       // turned back
      const float ones[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
      turn_factors<LAYOUT, 4>(c, s, ones, P, Q);
    }
    for (int part = 0; part < 3; ++part) {
      const int lo = part == 0 ? 0 : (part == 1 ? p.Hq : p.Hq + p.Hkv);
      const int heads = part == 0 ? p.Hq : p.Hkv;
      const int from = max(h_begin, lo), to = min(h_end, lo + heads);
      if (from >= to) continue;
      const int64_t head_step = static_cast<int64_t>(p.N) * p.d;
      const float* dz = (part == 0 ? p.dq : (part == 1 ? p.dk : p.dv)) +
                        (static_cast<int64_t>(b) * heads - lo) * head_step + static_cast<int64_t>(n) * p.d;
      const T* weight = static_cast<const T*>(part == 0 ? p.q_weight : p.k_weight);
      const bool nm = part < 2 && norm;
      const bool turned = LAYOUT != LAYOUT_NONE && part < 2 && m.rotated;
      uint64_t W[4] = {}, dW[4] = {};
      if (nm && m.on) {
        float w[8];
        load_weight<T, 4>(weight, m, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) W[k] = f2_pack(w[2 * k], w[2 * k + 1]);
      }
      for (int h0 = from; h0 < to; h0 += kRows) {
        Raw<float, 4> ga[kRows], gb[kRows];
        Raw<T, 4> xa[kRows], xb[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          ga[u].zero(), gb[u].zero(), xa[u].fill(pad), xb[u].fill(pad);
          if (m.on && live && h0 + u < to) {
            const float* src = dz + (h0 + u) * head_step;
            ga[u].load(src + m.a);
            gb[u].load(src + m.b);
            if (nm) {
              xa[u].load(row0 + (h0 + u) * p.d + m.a);
              xb[u].load(row0 + (h0 + u) * p.d + m.b);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          uint64_t g[4], dy[4];
          ga[u].pairs(g);
          gb[u].pairs(g + 2);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dy[k] = turned ? f2_fma(P[k], g[k], f2_mul(Q[k], partner<LAYOUT, 4>(g, k))) : g[k];
          if (nm) {
            uint64_t x[4], t[4];
            xa[u].pairs(x);
            xb[u].pairs(x + 2);
            uint64_t ss = 0, sd = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              t[k] = f2_mul(dy[k], x[k]);
              ss = f2_fma(x[k], x[k], ss);
              sd = f2_fma(t[k], W[k], sd);
            }
            float s0, s1, d0, d1;
            f2_unpack(ss, s0, s1);
            f2_unpack(sd, d0, d1);
            const float r = rsqrtf(row_sum<GS>(s0 + s1) * p.inv_d + p.eps);
            const float k2 = -r * (r * row_sum<GS>(d0 + d1)) * p.inv_d;      // r^3 may leave fp32, this only with r^2
            const uint64_t rr = f2_pack(r, r), kk = f2_pack(k2, k2);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              dW[k] = f2_fma(t[k], rr, dW[k]);
              dy[k] = f2_mul(f2_fma(x[k], kk, f2_mul(dy[k], W[k])), rr);
            }
          }
          if (m.on && live && h0 + u < to) {
            T* dst = drow0 + (h0 + u) * p.d;
            store_pairs<T, 4>(dst + m.a, dy);
            store_pairs<T, 4>(dst + m.b, dy + 2);
          }
        }
      }
      if (nm && live) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float4* mine = &acc[part][i][threadIdx.x];
          const float4 t = *mine;
          float a, b2, c2, d2;
          f2_unpack(dW[2 * i], a, b2);
          f2_unpack(dW[2 * i + 1], c2, d2);
          *mine = make_float4(t.x + a, t.y + b2, t.z + c2, t.w + d2);
        }
      }
    }
  }
  if (!norm) return;
  __syncthreads();
  // thread = (weight, piece, lane of the row): its four channels over the groups in order
  for (int e = threadIdx.x; e < 4 * GS; e += kThreads) {
    const int w = e / (2 * GS), piece = e / GS % 2, le = e % GS;
    const Lane me = lane_channels<LAYOUT, 4>(le, p.d, p.rot);
    if (!me.on) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int g = 0; g < kTokens; ++g) {
      const float4 t = acc[w][piece][g * GS + le];
      v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
    }
    *reinterpret_cast<float4*>(p.dw_partial + static_cast<int64_t>(blockIdx.x) * 2 * p.d + w * p.d +
                               (piece ? me.b : me.a)) = v;
  }
}

// dw[e] = the blocks' partial sums, e over both weights' channels: 32 outputs
// a block, 32 threads each, added in 64 bits in a fixed order.
__global__ void __launch_bounds__(1024) dw_reduce_kernel(const float* __restrict__ partial, int blocks, int d,
                                                         float* __restrict__ dqw, float* __restrict__ dkw) {
  griddep_wait();
  __shared__ double part[32][33];
  const int col = threadIdx.x % 32, row = threadIdx.x / 32;
  const int e = blockIdx.x * 32 + col;
  double v = 0.0;
  if (e < 2 * d) {
#pragma unroll 8
    for (int k = row; k < blocks; k += 32) v += static_cast<double>(partial[static_cast<int64_t>(k) * 2 * d + e]);
  }
  part[row][col] = v;
  __syncthreads();
  // warp `row` takes output `row`: its lanes hold the 32 threads' sums
  v = part[col][row];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int out = blockIdx.x * 32 + row;
  if (col == 0 && out < 2 * d) (out < d ? dqw[out] : dkw[out - d]) = static_cast<float>(v);
}

template <typename T, int GS, int LAYOUT, int E>
cudaError_t launch_fwd(NormRopeArgs p, int num_sms, cudaStream_t st) {
  constexpr int kTokens = kThreads / GS;
  const int64_t tiles = (static_cast<int64_t>(p.B) * p.N + kTokens - 1) / kTokens;
  const int H = p.Hq + 2 * p.Hkv;
  // heads of one token are split over blocks only while the token tiles alone leave multiprocessors without two
  // blocks: each split forms the angles again
  int runs = 1;
  while (runs < H && tiles * runs < 2 * num_sms) runs *= 2;
  p.head_run = (H + runs - 1) / runs;
  return launch_dependent(fwd_kernel<T, GS, LAYOUT, E>,
                          dim3(static_cast<unsigned>(tiles), (H + p.head_run - 1) / p.head_run), dim3(kThreads), 0, st,
                          p);
}

template <typename T, int GS, int LAYOUT>
cudaError_t launch(NormRopeArgs p, bool bwd, int num_sms, cudaStream_t st) {
  constexpr int kTokens = kThreads / GS;
  const int64_t tiles = (static_cast<int64_t>(p.B) * p.N + kTokens - 1) / kTokens;
  const int H = p.Hq + 2 * p.Hkv;
  if (!bwd) {
    // 16-byte pieces of bf16 where the widths allow them
    if constexpr (sizeof(T) == 2)
      if (p.d % 16 == 0 && p.rot % 16 == 0) return launch_fwd<T, GS / 2, LAYOUT, 8>(p, num_sms, st);
    return launch_fwd<T, GS, LAYOUT, 4>(p, num_sms, st);
  }
  // units of as many heads as a lane has in flight, fewer where that leaves blocks without work (single tokens)
  const int slots = norm_rope_bwd_blocks(num_sms);
  p.head_run = bwd_rows<T>();
  while (p.head_run > 1 && tiles * ((H + p.head_run - 1) / p.head_run) < slots) --p.head_run;
  const int64_t items = tiles * ((H + p.head_run - 1) / p.head_run);
  const int grid = static_cast<int>(items < slots ? items : slots);
  cudaError_t e = launch_dependent(bwd_kernel<T, GS, LAYOUT>, dim3(grid), dim3(kThreads), 0, st, p);
  if (e != cudaSuccess || p.q_weight == nullptr) return e;
  return launch_dependent(dw_reduce_kernel, dim3((2 * p.d + 31) / 32), dim3(1024), 0, st, p.dw_partial, grid, p.d,
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

int norm_rope_bwd_blocks(int num_sms) { return nrope::kBwdCtasPerSm * num_sms; }

cudaError_t launch_norm_rope(const NormRopeArgs& a, bool bf16, bool bwd, int num_sms, cudaStream_t st) {
  return bf16 ? nrope::by_width<__nv_bfloat16>(a, bwd, num_sms, st) : nrope::by_width<float>(a, bwd, num_sms, st);
}

}  // namespace bsa
