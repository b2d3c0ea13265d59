// attn_decode_quant.cu -- decode attention over the quantised paged cache
// (quant_cache.cu): one query token per sequence, each sequence its own
// length, over the kept blocks of a list or over every block.
//
// Formula.  A key is K_t 2^a_t, a value V_t 2^b_t (K, V rows of e4m3 codes,
// a, b the row's exponents).  With x_t = (q . K_t) 2^a_t scale log2(e) and
// y_t = x_t + b_t, any reference M >= about max y:
//   w_t = 2^(y_t - M),  O = sum w_t V_t,  l = sum 2^(x_t - M),  o = O / l,
// so the value's exponent rides in the softmax weight and the matrix product
// takes the codes as they are.  lse = ln2 (M + log2 l).
//
// Bound: memory.  A key and its value are 2 (d + 1) bytes and 4 d operations
// for each of at most 16 heads; the cache's own bytes, read once per KV head
// for all its query heads, are the floor.  So the design keeps loads in
// flight and spends few instructions a byte:
//   - a warp takes 16 keys at a time through two stages of its own: asynchronous
//     copies bring the next 4 KB while it works on a chunk and run on across the
//     rows of its range; no barrier and no block-wide wait stands in the loop.
//   - the codes become fp16 pairs by one conversion each (exact), and the
//     products run on m16n8k16 matrix instructions with the keys (then the
//     channels) as the 16 rows and eight query heads as the 8 columns.  The
//     order of the contracted index is free as long as both operands agree,
//     so each lane's share is what 16-byte reads of a stage bring: channels for
//     q . K; for V, lanes pair two keys' bytes and number the channels as they
//     hold them.  Tensor-memory instructions would need the codes split from
//     their rows' exponents across lanes and a block-wide exchange of maxima
//     for every 128 keys, at twice the keys a second of the bf16 kernel, for
//     a part that is not the bound: the matrix unit is 20% busy.
//   - M moves only when some y passes it by 2^7 (one vote a step; M starts at
//     the first maximum): w is scaled by 2^8, so it stays within fp16 and keeps
//     its 11 bits down to 2^-22 of the largest.
// w is rounded to fp16 for the product, the matrix unit's type that takes the
// codes exactly: at most 2^-11 of w, an eighth of the output's own rounding to
// bf16, or 2^-33 of the largest w.  l sums its terms unrounded; logits, O and l
// are fp32.
//
// Work split: the rows' list positions are laid end to end, each sequence
// with the blocks it has, and cut into equal ranges, one per team of warps: a
// block of threads is one team, or two or four where there are many rows, so
// that a team has about a row and another team's loads fill the time in which
// it joins its warps.  A range that holds a whole row writes its output; a row
// cut by range borders leaves one partial record (M, l, O) per range, at most
// two a team, and the second kernel joins them.
//
// 16 ragged sequences of 8 KV heads, 32 query heads: every block (2.5 GB) 382 to
// 393 us (95 to 98% of the copy rate, by the clock under the power cap), 97 kept
// blocks 37.1 to 39.0 us (80 to 84%), of which some 4.5 pass before the first
// keys are there (list, table, keys, one after the other, with cold code) and
// 1.3 in the join; one sequence of 30000 tokens 17.0 to 18.7 us, of 4001 11.0 to
// 11.9.  d = 64: every block 201 us (94%), 97 kept blocks 23.3 us (67%).  128
// query heads: every block 473 to 482 us (78%; d = 64 271 us, 70%), 97 kept
// blocks 47.8 us (65%).
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace bsa {
namespace qdecode {

constexpr float kLift = 8.0f;        // weights are 2^(y - M + 8)
constexpr float kHeadroom = 7.0f;    // M moves when y > M + 7: weights stay below 2^15
// A key's term of l is u = 2^(x - M + 8 + 16) and its weight u 2^(b - 16): with the
// 16, u stays normal 31 octaves below its largest for any b.  For M an exponent
// byte counts as at least 56, so u is at most 2^102 and 2^25 of them stay finite,
// whatever rows of zeros (byte 10) stand before others.  Rows below 56 (values
// under 2^-62) weigh less than M would let them, down to fp16's subnormals: an
// error of o under 2^-94, absolute.
constexpr int kDeep = 16;
constexpr uint32_t kLeastExp = 56u;

// NB = sets of eight query heads a warp carries; one block an SM: 16 warps of
// two stages (three stages: 97 kept blocks x 16 sequences 41.6 us against 40.2),
// or, where two sets (groups of 9 to 16 heads) take more registers, 12 (128 query
// heads, every block, us: 12 warps 482, 8 warps of six stages 507, 16 with the
// queries in shared memory 486, slower in short calls; four stages 483).
__host__ __device__ constexpr int warps(int NB) { return NB == 1 ? 16 : 12; }
constexpr int kStages = 2;
// a stage: 16 key rows, 16 value rows, their exponent bytes
__host__ __device__ constexpr int stage_bytes(int D) { return 2 * 16 * D + 32; }

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
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// a / b, with the short division wherever 32 bits hold them: a 64-bit one takes about 0.3 us of a start-up or a switch
// of rows.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
// `total` positions cut into at most `most` ranges, none of them empty: range i is [i total / count,
// (i+1) total / count), so borders of rows of equal length stay borders.
struct Cut {
  int64_t total, each;
  int rest, count;
  __device__ __forceinline__ Cut(int64_t all, int most) : total(all) {
    count = static_cast<int>(min(static_cast<int64_t>(most), total));
    each = count > 0 ? quotient(total, count) : 0;
    rest = static_cast<int>(total - each * count);
  }
  __device__ __forceinline__ int64_t begin(int i) const {
    return i * each + quotient(static_cast<int64_t>(i) * rest, count);
  }
  __device__ __forceinline__ int holds(int64_t x) const {      // the range of position x
    return static_cast<int>(quotient((x + 1) * count + total - 1, total)) - 1;
  }
};
__device__ __forceinline__ void team_sync(int team, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(threads) : "memory");
}

// Without a list, pre[b] = blocks of the sequences before b, b <= B: a
// sequence has as many positions (of one KV head) as it has blocks.  With one
// every sequence has list_len positions and nothing is read for the plan.
template <int kWarps>
__device__ __forceinline__ void plan_positions(const QuantDecodeArgs& p, int* pre, int* warp_sums) {
  constexpr int kThreads = 32 * kWarps;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + tid;
    int w = 0;
    if (b < p.B) {
      const int len = p.lens ? min(max(p.lens[b], 0), p.nb * 64) : p.nb * 64;
      w = (len + 63) >> 6;
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

// Where 16-byte piece q of a staged row stands, q ^ swizzle(row): eight lanes
// that read together then meet eight different 16-byte columns.  Keys: two
// neighbouring rows, four pieces each; values: rows 2c, two pieces each (one,
// shared by two lanes, where a row is 64 bytes).
template <int D>
__device__ __forceinline__ int k_swizzle(int row) {
  return D == 128 ? (row & 1) * 4 : 0;
}
template <int D>
__device__ __forceinline__ int v_swizzle(int row) {
  return D == 128 ? (row & 6) : ((row >> 2) & 1) * 2;
}

// One row's stretch of list positions inside a range.
struct Item {
  int b, g, w, t0, t1;
  int64_t next;      // first position behind it
};

// The item that begins at position x < hi; b: a sequence not behind x's.
__device__ __forceinline__ Item item_at(const QuantDecodeArgs& p, const int* pre, int64_t x, int64_t hi, int b) {
  Item it;
  int64_t row0;
  if (p.idx) {
    it.w = p.list_len;
    const int bg = static_cast<int>(quotient(x, it.w));
    it.b = bg / p.Hkv;
    it.g = bg - it.b * p.Hkv;
    row0 = static_cast<int64_t>(bg) * it.w;
  } else {
    while (x >= static_cast<int64_t>(pre[b + 1]) * p.Hkv) ++b;     // passes sequences without a block too
    it.b = b;
    it.w = pre[b + 1] - pre[b];
    const int64_t seq0 = static_cast<int64_t>(pre[b]) * p.Hkv;
    it.g = static_cast<int>(quotient(x - seq0, it.w));
    row0 = seq0 + static_cast<int64_t>(it.g) * it.w;
  }
  it.t0 = static_cast<int>(x - row0);
  it.t1 = static_cast<int>(min(hi - row0, static_cast<int64_t>(it.w)));
  it.next = row0 + it.t1;
  return it;
}

// Where channel pair (r * D/8 + 2 mb) of query head 2c or 2c+1 stands among a
// head's pairs while warps are joined: a warp's stores fill the banks.
template <int D>
__device__ __forceinline__ int pair_at(int r, int mb, int c) {
  return r * (D / 16) + (mb ^ ((2 * c + ((r >> 1) & 1)) & (D / 16 - 1)));
}

template <int D, int NB>
__global__ void __launch_bounds__(32 * warps(NB), 1) decode_kernel(const QuantDecodeArgs p) {
  constexpr int kWarps = warps(NB), kThreads = 32 * kWarps;
  constexpr int KH = D / 64;        // 64-byte halves of a row
  constexpr int KS = D / 16;        // k-steps of q . K
  constexpr int MB = D / 16;        // 16-channel row blocks of O
  constexpr int VW = D / 32;        // 32-bit words of a V row per lane
  constexpr int R = kStages;
  constexpr int SB = stage_bytes(D);
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ float sm_m[kWarps][8 * NB], sm_l[kWarps][8 * NB];
  __shared__ int sm_slot[kWarps], warp_sums[kWarps];
  int* pre = reinterpret_cast<int*>(smem_raw + kWarps * R * SB);
  griddep_wait();   // lists, lengths and the cache come from the kernels launched before
  if (p.idx == nullptr) {
    plan_positions<kWarps>(p, pre, warp_sums);
    if (blockIdx.x == 0)
      for (int b = threadIdx.x; b <= p.B; b += kThreads) p.pre[b] = pre[b];
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int G = p.Hq / p.Hkv;
  const int64_t total = static_cast<int64_t>(p.idx ? p.B * p.list_len : pre[p.B]) * p.Hkv;
  // teams: the first of every block, then the second of every block, ...
  const int team_warps = p.team_warps, team = warp / team_warps, tw = warp - team * team_warps;
  const int range = team * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
  const Cut cut(total, p.num_ranges);
  if (range >= cut.count) return;
  const int64_t x = cut.begin(range), hi = cut.begin(range + 1);
  int b_first = 0;
  if (p.idx == nullptr) {   // the sequence of position x: the last b with pre[b] * Hkv <= x
    int hi_b = p.B;
    while (hi_b - b_first > 1) {
      const int mid = (b_first + hi_b) / 2;
      if (static_cast<int64_t>(pre[mid]) * p.Hkv <= x) b_first = mid; else hi_b = mid;
    }
  }

  // ---- the loading side, R chunks ahead of the other: an item's chunks of 16 keys go to the team's warps in
  // turn, a warp looks 32 of its own up at once (one a lane), and runs on into the team's next items by itself
  uint8_t* ring = smem_raw + warp * R * SB;
  const uint32_t ring_u32 = smem_u32(ring);
  Item li = item_at(p, pre, x, hi, b_first);   // item being loaded
  Item it = li;                                 // item being worked on
  int l_no = 0;                                 // its number
  int l_base = tw - 32 * team_warps;            // first chunk of the batch held
  int turn = 0;                                 // the warp that takes the item's first chunk: dealt on across items
  int l_len = 0;
  unsigned l_left = 0u;                         // lanes whose chunk is still to be taken
  int my_row = 0, my_n = 0;                     // the lane's chunk: row of 16 in the pools, keys that count
  int meta = -1;                                // lane s: stage s's item number * 32 + keys, or -1
  auto seq_len = [&](int b) { return p.lens ? min(max(__ldg(p.lens + b), 0), p.nb * 64) : p.nb * 64; };
  l_len = seq_len(li.b);
  auto refill = [&](int slot) {
    bool have = true;
    while (l_left == 0u) {
      l_base += 32 * team_warps;
      if (l_base >= 4 * (li.t1 - li.t0)) {
        if (li.next >= hi) {
          have = false;
          l_base -= 32 * team_warps;
          break;
        }
        turn = (turn + 4 * (li.t1 - li.t0)) % team_warps;
        li = item_at(p, pre, li.next, hi, li.b);
        l_len = seq_len(li.b);
        ++l_no;
        l_base = tw - turn + (tw < turn ? team_warps : 0);
      }
      const int u = l_base + lane * team_warps;
      my_n = 0;
      if (u < 4 * (li.t1 - li.t0)) {
        const int t = li.t0 + (u >> 2);
        const int blk = p.idx ? __ldg(p.idx + (static_cast<int64_t>(li.b) * p.Hkv + li.g) * p.list_len + t) : t;
        const int pos = max(min(blk, p.nb), -1) * 64 + (u & 3) * 16;
        if (blk >= p.nb) {
          atomicOr(p.status, BSA_DEV_BAD_INDEX);
        } else if (blk >= 0 && pos < l_len) {
          const int page = __ldg(p.table + static_cast<int64_t>(li.b) * p.table_stride + blk);
          if (page < 0 || page >= p.num_pages) {
            atomicOr(p.status, BSA_DEV_BAD_INDEX);
          } else {
            my_n = min(16, l_len - pos);
            my_row = (page * p.Hkv + li.g) * 4 + (u & 3);
          }
        }
      }
      l_left = __ballot_sync(0xffffffffu, my_n > 0);
    }
    int said = -1;
    if (have) {
      const int src = __ffs(l_left) - 1;
      l_left &= l_left - 1;
      const int row = __shfl_sync(0xffffffffu, my_row, src);
      said = l_no * 32 + __shfl_sync(0xffffffffu, my_n, src);
      const uint32_t dst = ring_u32 + slot * SB;
      const uint8_t* k = p.k_pool + static_cast<int64_t>(row) * (16 * D) + lane * 16;
      const uint8_t* v = p.v_pool + static_cast<int64_t>(row) * (16 * D) + lane * 16;
      // 512 bytes a step, whole rows: the step changes the row by a multiple of 4, so the lane's place in it is fixed
      // but for the values' swizzle, which takes bit 2 of the row
      constexpr int PR = D / 16, kStep = 32 / PR;      // 16-byte pieces of a row, rows of a step
      const int rr = lane / PR, q = lane % PR;
      const uint32_t kd = dst + rr * D + (q ^ k_swizzle<D>(rr)) * 16;
      const uint32_t vd0 = rr * D + (q ^ v_swizzle<D>(rr)) * 16, vd1 = rr * D + (q ^ v_swizzle<D>(rr + 4)) * 16;
#pragma unroll
      for (int i = 0; i < PR / 2; ++i) {
        cp_async16(kd + i * 512, k + i * 512);
        cp_async16(dst + 16 * D + i * 512 + ((i * kStep) & 4 ? vd1 : vd0), v + i * 512);
      }
      if (lane < 2) cp_async16(dst + 32 * D + lane * 16, (lane ? p.v_exp : p.k_exp) + static_cast<int64_t>(row) * 16);
    }
    cp_async_commit();
    if (lane == slot) meta = said;
  };
  // the item's query heads as loaded, asked for before its keys or while the warps of the item before are joined
  uint32_t qf[NB][KS][2];
  auto load_q = [&](const Item& i) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int h = nb * 8 + r;
      const __nv_bfloat16* qrow = p.q + (static_cast<int64_t>(i.b) * p.Hq + i.g * G + h) * D;
#pragma unroll
      for (int hf = 0; hf < KH; ++hf)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 v = h < G ? __ldg(reinterpret_cast<const uint4*>(qrow + hf * 64 + c * 16 + 8 * j))
                                : make_uint4(0, 0, 0, 0);
          qf[nb][hf * 4 + 2 * j][0] = v.x;
          qf[nb][hf * 4 + 2 * j][1] = v.y;
          qf[nb][hf * 4 + 2 * j + 1][0] = v.z;
          qf[nb][hf * 4 + 2 * j + 1][1] = v.w;
        }
    }
  };
  load_q(it);
  for (int s = 0; s < R; ++s) refill(s);

  int head = 0;               // stage to be taken next
  for (int no = 0;; ++no) {
    // ---- the group's query heads, scaled by a power of two into fp16: a head's largest value goes to
    // [2^10, 2^11), smaller ones keep their eight bits down to 2^-25 of it
    float qs[NB][2];        // logit factors of heads 2c, 2c+1 of each set
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float amax = 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(qf[nb][k][i] << 16)),
                                   fabsf(__uint_as_float(qf[nb][k][i] & 0xFFFF0000u))));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int E = max(static_cast<int>(__float_as_uint(amax) >> 23), 11);
      const float up = __uint_as_float(static_cast<uint32_t>(264 - E) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qf[nb][k][i] = pack_f16x2(__uint_as_float(qf[nb][k][i] << 16) * up,
                                    __uint_as_float(qf[nb][k][i] & 0xFFFF0000u) * up);
      const float down = __uint_as_float(static_cast<uint32_t>(E - 10) << 23) * p.scale_log2;
      qs[nb][0] = __shfl_sync(0xffffffffu, down, (2 * c) * 4);
      qs[nb][1] = __shfl_sync(0xffffffffu, down, (2 * c + 1) * 4);
    }

    float M[NB][2], O[NB][MB][4];
    uint64_t l[NB];        // of two heads
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      M[nb][0] = M[nb][1] = -INFINITY;
      l[nb] = 0ull;
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) O[nb][m][i] = 0.0f;
    }
    int spare = -1;        // the item's last stage, kept back for the join
    for (;;) {
      const int said = __shfl_sync(0xffffffffu, meta, head);
      if (said < 0 || (said >> 5) != no) break;
      if (spare >= 0) refill(spare);
      const int n = said & 31;
      cp_async_wait_group<R - 1>();
      __syncwarp();
      const uint8_t* st = ring + head * SB;
      // ---- S = K q^T: rows r, r+8 x heads 2c, 2c+1
      float S[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[nb][0] = S[nb][1] = S[nb][2] = S[nb][3] = 0.0f;
#pragma unroll
      for (int hf = 0; hf < KH; ++hf) {
        const uint4 ka = *reinterpret_cast<const uint4*>(st + r * D + ((hf * 4 + c) ^ k_swizzle<D>(r)) * 16);
        const uint4 kb = *reinterpret_cast<const uint4*>(st + (r + 8) * D + ((hf * 4 + c) ^ k_swizzle<D>(r + 8)) * 16);
        const uint32_t a[4] = {ka.x, ka.y, ka.z, ka.w};
        const uint32_t e[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = cvt_e4m3x2(a[i]), a1 = cvt_e4m3x2(e[i]), a2 = cvt_e4m3x2(a[i] >> 16),
                         a3 = cvt_e4m3x2(e[i] >> 16);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            mma16816(S[nb], a0, a1, a2, a3, qf[nb][hf * 4 + i][0], qf[nb][hf * 4 + i][1]);
        }
      }
      // ---- weights
      float kf[2], vf[2], vb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = r + 8 * i;
        uint32_t ke = st[32 * D + key], ve = st[32 * D + 16 + key];
        if (n < 16 && key >= n) ke = ve = 127u;     // may hold anything
        kf[i] = __uint_as_float(ke << 23);
        vf[i] = __uint_as_float((max(ve, static_cast<uint32_t>(kDeep)) - kDeep) << 23);
        vb[i] = __uint_as_float(0x4B000000u | max(ve, kLeastExp)) - 8388735.0f;      // - 127, through 2^23
      }
      uint32_t wb[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        uint64_t yy[2];        // a key's logits of two heads
        bool high = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // the factors first: S 2^a alone may leave fp32 where the logit does not (large keys, small queries); their
          // product leaves it only for logits past 2^95 or under 2^-99 (2^-33 <= |S| < 2^27)
          yy[i] = f2_mul(f2_pack(S[nb][2 * i], S[nb][2 * i + 1]), f2_mul(f2_pack(kf[i], kf[i]), f2_pack(qs[nb][0], qs[nb][1])));
          if (n < 16 && r + 8 * i >= n) yy[i] = f2_pack(-INFINITY, -INFINITY);
          float y0, y1;
          f2_unpack(f2_add(yy[i], f2_pack(vb[i], vb[i])), y0, y1);
          high |= y0 > M[nb][0] + kHeadroom || y1 > M[nb][1] + kHeadroom;
        }
        if (__any_sync(0xffffffffu, high)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float ya[2], yb[2];
            f2_unpack(yy[0], ya[0], ya[1]);
            f2_unpack(yy[1], yb[0], yb[1]);
            float t = fmaxf(ya[h] + vb[0], yb[h] + vb[1]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
            const float m_new = fmaxf(M[nb][h], t);
            const float root = (m_new == -INFINITY) ? 1.0f : fast_exp2(0.5f * (M[nb][h] - m_new));
            M[nb][h] = m_new;
            const uint64_t rr = h ? f2_pack(1.0f, root) : f2_pack(root, 1.0f);
            l[nb] = f2_mul(f2_mul(l[nb], rr), rr);
            const float a = root * root;
#pragma unroll
            for (int m = 0; m < MB; ++m) {
              O[nb][m][h] *= a;
              O[nb][m][2 + h] *= a;
            }
          }
        }
        const float ref0 = (M[nb][0] == -INFINITY) ? 0.0f : kLift + kDeep - M[nb][0];
        const float ref1 = (M[nb][1] == -INFINITY) ? 0.0f : kLift + kDeep - M[nb][1];
        float wgt[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float e0, e1;
          f2_unpack(f2_add(yy[i], f2_pack(ref0, ref1)), e0, e1);
          const uint64_t u = f2_pack(fast_exp2(e0), fast_exp2(e1));
          l[nb] = f2_add(l[nb], u);
          f2_unpack(f2_mul(u, f2_pack(vf[i], vf[i])), wgt[2 * i], wgt[2 * i + 1]);
        }
        // keys x heads -> heads x keys: the B operand of O^T = V^T w
        wb[nb][0] = transpose8x8(pack_f16x2(wgt[0], wgt[1]));
        wb[nb][1] = transpose8x8(pack_f16x2(wgt[2], wgt[3]));
      }
      uint32_t vr[4][VW];       // rows 2c, 2c+1, 2c+8, 2c+9: D/8 bytes at r * D/8
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 2 * c + (i & 1) + 8 * (i >> 1);
        const uint8_t* src = st + 16 * D + row * D;
        if constexpr (D == 128) {
          const uint4 t = *reinterpret_cast<const uint4*>(src + (r ^ v_swizzle<D>(row)) * 16);
          vr[i][0] = t.x, vr[i][1] = t.y, vr[i][2] = t.z, vr[i][3] = t.w;
        } else {
          const uint2 t = *reinterpret_cast<const uint2*>(src + ((r >> 1) ^ v_swizzle<D>(row)) * 16 + (r & 1) * 8);
          vr[i][0] = t.x, vr[i][1] = t.y;
        }
      }
      if (n < 16) {   // rows past the sequence may hold anything: a zero weight does not silence a NaN
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (2 * c + (i & 1) + 8 * (i >> 1) >= n) {
#pragma unroll
            for (int k = 0; k < VW; ++k) vr[i][k] = 0u;
          }
      }
#pragma unroll
      for (int k = 0; k < VW; ++k) {
        // bytes of two keys side by side: channels (0,1) and (2,3) of this word
        const uint32_t lo01 = __byte_perm(vr[0][k], vr[1][k], 0x5140), lo23 = __byte_perm(vr[0][k], vr[1][k], 0x7362);
        const uint32_t hi01 = __byte_perm(vr[2][k], vr[3][k], 0x5140), hi23 = __byte_perm(vr[2][k], vr[3][k], 0x7362);
        const uint32_t a[2][4] = {{cvt_e4m3x2(lo01), cvt_e4m3x2(lo01 >> 16), cvt_e4m3x2(hi01), cvt_e4m3x2(hi01 >> 16)},
                                  {cvt_e4m3x2(lo23), cvt_e4m3x2(lo23 >> 16), cvt_e4m3x2(hi23), cvt_e4m3x2(hi23 >> 16)}};
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            mma16816(O[nb][2 * k + u], a[u][0], a[u][1], a[u][2], a[u][3], wb[nb][0], wb[nb][1]);
      }
      __syncwarp();
      spare = head;
      head = head + 1 == R ? 0 : head + 1;
    }

    const bool more = it.next < hi;
    Item next = it;
    if (more) {
      next = item_at(p, pre, it.next, hi, it.b);
      load_q(next);
    }

    // ---- join the warps, then write the row or its partial record; a warp's O waits in its spare stage
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float ls[2];
      f2_unpack(l[nb], ls[0], ls[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) ls[h] += __shfl_xor_sync(0xffffffffu, ls[h], o);
        // a NaN logit leaves M as it is; without another key the row must still not pass for an empty one
        if (M[nb][h] == -INFINITY && ls[h] != ls[h]) M[nb][h] = 0.0f;
        if (r == 0) {
          sm_m[warp][nb * 8 + 2 * c + h] = M[nb][h];
          sm_l[warp][nb * 8 + 2 * c + h] = ls[h];
        }
      }
    }
    if (lane == 0) sm_slot[warp] = spare;
    const bool whole = it.t0 == 0 && it.t1 == it.w;
    const int slot = it.t0 > 0 ? 0 : 1;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (spare >= 0) {
        float2* mine = reinterpret_cast<float2*>(ring + spare * SB);
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            mine[(2 * c + h) * (D / 2) + pair_at<D>(r, m, c)] = make_float2(O[nb][m][h], O[nb][m][2 + h]);
      }
      team_sync(team, 32 * team_warps);
      // a warp takes 32 channel pairs of a query head: lane k (of either half) holds warp k's share, the largest M
      // and the sum of l come by exchange
      const int units = min(8, G - nb * 8) * (D / 64), w0 = team * team_warps, mate = lane & 15;
      for (int unit = tw; unit < units; unit += team_warps) {
        const int h = unit / (D / 64), pr = unit % (D / 64) * 32 + lane;         // query head of the set, channel pair
        const int at = h * (D / 2) + pair_at<D>(pr / (D / 16), pr % (D / 16), h >> 1);
        const float m_k = mate < team_warps ? sm_m[w0 + mate][nb * 8 + h] : -INFINITY;
        float mx = m_k;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        float f = 0.0f, L = 0.0f;
        int from = 0;
        if (m_k != -INFINITY) {      // else a warp without a key: it may have no spare stage
          const float root = fast_exp2(0.5f * (m_k - mx));
          f = root * root;
          L = root * sm_l[w0 + mate][nb * 8 + h] * root;
          from = ((w0 + mate) * R + sm_slot[w0 + mate]) * SB;
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        float o0 = 0.0f, o1 = 0.0f;
#pragma unroll 8
        for (int k = 0; k < team_warps; ++k) {
          const float fk = __shfl_sync(0xffffffffu, f, k);
          const int from_k = __shfl_sync(0xffffffffu, from, k);
          float2 v = make_float2(0.0f, 0.0f);
          if (fk != 0.0f) v = reinterpret_cast<const float2*>(smem_raw + from_k)[at];
          o0 += fk * v.x;
          o1 += fk * v.y;
        }
        const int64_t orow = static_cast<int64_t>(it.b) * p.Hq + it.g * G + nb * 8 + h;
        if (whole) {
          const float inv = (mx == -INFINITY) ? 0.0f : static_cast<float>(1 << kDeep) / L;
          reinterpret_cast<uint32_t*>(p.o + orow * D)[pr] = pack_bf16x2(o0 * inv, o1 * inv);
          if (p.lse && pr == 0)
            p.lse[orow] = (mx == -INFINITY) ? -INFINITY : (mx - (kLift + kDeep) + log2f(L)) * 0.69314718055994530942f;
        } else {
          float* rec = p.partial + ((static_cast<int64_t>(range) * 2 + slot) * G + nb * 8 + h) * (D + 4);
          *reinterpret_cast<float2*>(rec + 4 + 2 * pr) = make_float2(o0, o1);
          if (pr == 0) {
            rec[0] = mx;
            rec[1] = L;
          }
        }
      }
      team_sync(team, 32 * team_warps);
    }
    if (!more) break;
    if (spare >= 0) refill(spare);
    it = next;
  }
  cp_async_wait_group<0>();
}

// One block per (sequence, query head): rows cut by range borders are joined
// from their records, rows without a key become zero; rows that one range
// held are complete already.  Latency is all: eight records (M, l and this
// thread's channel of O) are asked for at once and folded into a running
// (M, l, O), and where a row has many records PARTS threads a channel share
// them.
template <int D, int PARTS>
__global__ void __launch_bounds__(D * PARTS) combine_kernel(const QuantDecodeArgs p) {
  griddep_wait();
  __shared__ float part_m[PARTS], part_l[PARTS], part_o[PARTS][D];
  const int G = p.Hq / p.Hkv;
  const int b = blockIdx.x / p.Hq, hq = blockIdx.x - b * p.Hq;
  const int g = hq / G, h = hq - g * G;
  const int ch = threadIdx.x % D, part = threadIdx.x / D;
  const int64_t orow = blockIdx.x;
  const int before = p.idx ? b * p.list_len : p.pre[b], w = p.idx ? p.list_len : p.pre[b + 1] - before;
  const int64_t total = static_cast<int64_t>(p.idx ? p.B * p.list_len : p.pre[p.B]) * p.Hkv;
  if (w == 0) {
    if (part == 0) p.o[orow * D + ch] = __float2bfloat16_rn(0.0f);
    if (p.lse && threadIdx.x == 0) p.lse[orow] = -INFINITY;
    return;
  }
  const Cut cut(total, p.num_ranges);
  const int64_t x0 = static_cast<int64_t>(before) * p.Hkv + static_cast<int64_t>(g) * w;
  const int first = cut.holds(x0), n = cut.holds(x0 + w - 1) - first + 1;
  if (n == 1) return;
  // the row begins inside range `first` (its record 1) and goes on in the next ones (their records 0)
  const float* rec = p.partial + (static_cast<int64_t>(first) * 2 * G + h) * (D + 4);
  const int step = 2 * G * (D + 4);
  float M = -INFINITY, L = 0.0f, acc = 0.0f;
  for (int k0 = part; k0 < n; k0 += 8 * PARTS) {
    float2 ml[8];
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = k0 + i * PARTS;
      const float* at = rec + (k == 0 ? G * (D + 4) : static_cast<int64_t>(k) * step);
      ml[i] = k < n ? *reinterpret_cast<const float2*>(at) : make_float2(-INFINITY, 0.0f);
      o[i] = k < n ? at[4 + ch] : 0.0f;
    }
    float m_new = M;
#pragma unroll
    for (int i = 0; i < 8; ++i) m_new = fmaxf(m_new, ml[i].x);
    if (m_new == -INFINITY) continue;
    const float root = exp2f(0.5f * (M - m_new));
    L = L * root * root;
    acc *= root * root;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = exp2f(0.5f * (ml[i].x - m_new));     // 0 where the record is empty
      L += f * ml[i].y * f;
      acc += f * f * o[i];
    }
    M = m_new;
  }
  if constexpr (PARTS > 1) {
    if (ch == 0) {
      part_m[part] = M;
      part_l[part] = L;
    }
    part_o[part][ch] = acc;
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int k = 1; k < PARTS; ++k) M = fmaxf(M, part_m[k]);
    L = acc = 0.0f;
    if (M != -INFINITY) {
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        const float f = exp2f(0.5f * (part_m[k] - M));
        L += f * part_l[k] * f;
        acc += f * f * part_o[k][ch];
      }
    }
  }
  p.o[orow * D + ch] = __float2bfloat16_rn(M == -INFINITY ? 0.0f : acc * (static_cast<float>(1 << kDeep) / L));
  if (p.lse && ch == 0) p.lse[orow] = (M == -INFINITY) ? -INFINITY : (M - (kLift + kDeep) + log2f(L)) * 0.69314718055994530942f;
}

template <int D, int NB>
cudaError_t launch(const QuantDecodeArgs& a, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(warps(NB)) * kStages * stage_bytes(D) +
                      (a.idx ? 0 : (static_cast<size_t>(a.B) + 1) * sizeof(int));
  cudaError_t e = ensure_dynamic_smem<decode_kernel<D, NB>>(smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(decode_kernel<D, NB>, dim3(a.num_ctas), dim3(32 * warps(NB)), smem, st, a);
  if (e != cudaSuccess) return e;
  // rows of equal length on ranges of whole rows: every output is written
  if (a.idx && a.B * a.Hkv % a.num_ranges == 0) return cudaSuccess;
  // records a row: the ranges over the rows, on average; over one round of eight they are shared out
  if (a.num_ranges > 8 * a.B * a.Hkv) return launch_dependent(combine_kernel<D, 4>, dim3(a.B * a.Hq), dim3(4 * D), 0, st, a);
  return launch_dependent(combine_kernel<D, 1>, dim3(a.B * a.Hq), dim3(D), 0, st, a);
}

}  // namespace qdecode

// One team of all warps an SM, or, while there are more rows than teams, two or
// four smaller ones (33 kept blocks, us: 192 rows in two teams an SM 25.1, in one
// 28.8; 512 rows in four 52.1, in two 55.9); two also where rows of unknown
// lengths number more than half of the SMs (128 rows of 1.5K to 3K tokens 22.3 us,
// in one team an SM 24.4; 96 of 2K to 6K 25.9 and 26.7; at 64 rows they are even,
// 16.1 and 16.5): such rows are cut, and one team loads while the other joins.
// All multiprocessors take part (the whole cache of 16 sequences 387 to 390 us, on
// 7/8 of them 404 to 415).
// Ranges that end where rows end leave fewer records to join (97 kept blocks,
// us: 24 rows on 144 ranges 13.0, on 148 15.9; 48 on 144 18.0 and 21.2; 120 on
// 120 35.6 and 40.4; 128 on 128 37.3 to 37.9 and 41.1; 33 blocks, 256 rows on 256
// 27.4, on 296 31.4): from a list, where rows are equally long, as many ranges a
// row as fit the teams, or whole rows a range, if that keeps at least 4/5 of the
// teams busy.  With fewer busy it goes either way (80 rows on 80 33.1, on 148
// 29.2; 160 on 160 24.0, on 296 22.6; but 112 on 112 33.8, on 148 37.1).  Without a
// list only where a row has four ranges or more (32 rows of 15K to 30K tokens on
// 128 38.1, on 148 38.7; 8 rows on 144 12.9 and 15.7; 48 rows may gain or lose:
// its own length may be the only one).
QuantSplit quant_decode_split(int num_sms, int group, int rows, bool list, int forced) {
  const int NB = group > 8 ? 2 : 1;
  QuantSplit s;
  s.team_warps = qdecode::warps(NB);
  int teams = num_sms;
  if (forced > 0) {
    s.ranges = forced;
    s.ctas = forced;
    return s;
  }
  for (int half = 0; half < 2 && (rows > teams || (half == 0 && !list && 2 * rows > teams)); ++half) {
    s.team_warps /= 2;
    teams *= 2;
  }
  s.ranges = teams;
  const int each = (rows + teams - 1) / teams;          // rows a range, where there are more rows than teams
  const int even = rows <= teams ? rows * (teams / rows) : (rows + each - 1) / each;
  if (5 * even >= 4 * teams && (list || rows <= teams / 4)) s.ranges = even;
  s.ctas = s.ranges < num_sms ? s.ranges : num_sms;
  return s;
}

cudaError_t launch_attn_decode_quant(const QuantDecodeArgs& a, int d, cudaStream_t st) {
  if (a.Hq / a.Hkv > 8) return d == 64 ? qdecode::launch<64, 2>(a, st) : qdecode::launch<128, 2>(a, st);
  return d == 64 ? qdecode::launch<64, 1>(a, st) : qdecode::launch<128, 1>(a, st);
}

}  // namespace bsa
