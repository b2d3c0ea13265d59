// topk_lens.cu -- the decode selection for a batch whose sequences have
// their own lengths: row r of the scores belongs to sequence r / rows_per_len,
// which has n = ceil(len / block) blocks; candidates are the blocks j < n-1,
// the sequence's last block n-1 is always kept (SAS page, 推理 paragraph and
// 核心模块 3; "稀疏注意力" tutorial §5), and columns from it on do not count: in a
// growing cache they hold whatever was there before.
//
// One warp per row, the row's scores in its registers as bf16 pairs (rounded
// to nearest, which keeps their order up to ties).  A row is a few KB, so
// instructions count, not bytes: the bf16 threshold T (the largest with at
// least k scores >= T) is found by bisection of the 16-bit codes, 16 counts at
// one compare and one add for two scores, without a barrier or shared memory.
// Scores whose rounding is above T are kept; those that round to T (a few,
// as a rule) are listed and ranked by their full keys, or, where more than 32
// do, their lower key bits are bisected by 32 more counts over the row.
// Equal scores: the lower index first.  NaN compares with nothing, so it ranks
// last by itself.  The counts run over registers; then each lane takes 64
// consecutive columns (16 in short rows) from shared memory, keeps what is
// above T and what rounds to it as bits, and writes its kept columns behind
// those of the lanes before it: no step waits for another column's.  2048 rows
// of 1300 candidates: 11.7 us; a block of 256 threads a row with four 8-bit
// histograms took 21.2, one 12-bit histogram and a ranked list 22.3, ballots
// column by column instead of the lanes' bits 13.9.
#include "kernels.h"
#include "topk.cuh"

namespace bsa {
namespace topk_lens {

__device__ __forceinline__ __nv_bfloat162 as_pair(uint32_t v) { return *reinterpret_cast<__nv_bfloat162*>(&v); }
// A 16-bit code that orders as the bf16 values do, and back.
__device__ __forceinline__ uint32_t code_value(uint32_t code) { return code & 0x8000u ? code & 0x7FFFu : ~code & 0xFFFFu; }

template <int PAIRS>
__device__ __forceinline__ int count_ge(const uint32_t (&x)[PAIRS], uint32_t code) {
  const uint32_t t = code_value(code);
  const uint32_t both = t | (t << 16);
  __nv_bfloat162 acc[4];       // at most 256 each: exact in bf16
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = __hge2(as_pair(x[i]), as_pair(both));
#pragma unroll
  for (int p = 4; p < PAIRS; ++p) acc[p & 3] = __hadd2(acc[p & 3], __hge2(as_pair(x[p]), as_pair(both)));
  float c = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(acc[i]);
    c += f.x + f.y;
  }
  return __reduce_add_sync(0xffffffffu, static_cast<int>(c));
}

// Code of the row's largest score, below every number's where all are NaN.
template <int PAIRS>
__device__ __forceinline__ uint32_t code_max(const uint32_t (&x)[PAIRS]) {
  __nv_bfloat162 m = as_pair(x[0]);
#pragma unroll
  for (int p = 1; p < PAIRS; ++p) m = __hmax2(m, as_pair(x[p]));       // the other one, where one is NaN
  const uint32_t bits = *reinterpret_cast<const uint32_t*>(&m);
  uint32_t best = 0u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t v = (bits >> (16 * h)) & 0xFFFFu;
    const bool is_nan = (v & 0x7FFFu) > 0x7F80u;
    const uint32_t code = v & 0x8000u ? ~v & 0xFFFFu : v | 0x8000u;
    best = max(best, is_nan ? 0u : code);
  }
  return __reduce_max_sync(0xffffffffu, best);
}

// Pair p of lane l holds columns 64 p + 2 l and 64 p + 2 l + 1.
template <int PAIRS>
__global__ void __launch_bounds__(32) row_kernel(const float* __restrict__ scores, int ncols,
                                                 const int* __restrict__ lens, int rows_per_len, int block, int kb,
                                                 int* __restrict__ idx_out, int idx_stride,
                                                 int* __restrict__ count_out, uint32_t* __restrict__ status) {
  griddep_wait();   // the scores come from the kernel launched before
  const int lane = threadIdx.x;
  const int64_t r = blockIdx.x;
  const int len = lens[r / rows_per_len];
  const int n_all = len > 0 ? (len - 1) / block + 1 : 0;
  if (n_all > ncols && lane == 0) atomicOr(status, BSA_DEV_BAD_INDEX);
  const int n = min(n_all, ncols);
  const int ncand = max(n - 1, 0);
  const float* srow = scores + r * ncols;
  const float nan = __uint_as_float(0x7FFFFFFFu);
  constexpr int kChunk = PAIRS < 32 ? PAIRS : 32;          // pairs of a lane's columns, per round
  constexpr int kRounds = PAIRS / kChunk;
  __shared__ float2 xs[PAIRS * 32 + PAIRS * 32 / kChunk];   // a gap behind each chunk keeps the lanes' banks apart
  __shared__ uint32_t member_key[32];
  auto slot = [](int pair) { return pair + pair / kChunk; };
  uint32_t x[PAIRS];
  // 32 pairs at a time, asked for together: no branch stands between the loads
  const bool even = ncols % 2 == 0 && (reinterpret_cast<uintptr_t>(scores) & 7u) == 0;
  constexpr int kBatch = PAIRS < 32 ? PAIRS : 32;
#pragma unroll
  for (int p0 = 0; p0 < PAIRS; p0 += kBatch) {
    float2 v[kBatch];
    if (even) {
#pragma unroll
      for (int p = 0; p < kBatch; ++p) {
        const int j = 64 * (p0 + p) + 2 * lane;
        v[p] = j < ncand ? __ldg(reinterpret_cast<const float2*>(srow + j)) : make_float2(nan, nan);
      }
    } else {
#pragma unroll
      for (int p = 0; p < kBatch; ++p) {
        const int j = 64 * (p0 + p) + 2 * lane;
        v[p].x = j < ncand ? __ldg(srow + j) : nan;
        v[p].y = j + 1 < ncand ? __ldg(srow + j + 1) : nan;
      }
    }
#pragma unroll
    for (int p = 0; p < kBatch; ++p) {
      if (64 * (p0 + p) + 2 * lane + 1 >= ncand) v[p].y = nan;     // the row's next column, where it was read
      x[p0 + p] = pack_bf16x2(v[p].x, v[p].y);
      xs[slot(32 * (p0 + p) + lane)] = v[p];
    }
  }
  const int take = min(kb, ncand);
  // kept: scores that round above T; of those that round to T, full keys above `thresh`; of the keys equal to it the
  // first `ties`.  Code kNone stands below every number's: there the scores that "round to T" are the NaNs.
  constexpr uint32_t kNone = 0x007Eu;
  uint32_t t_code = 0xFFFFu, thresh = 0u;     // nothing is kept
  int ties = 0, remaining = 0, members = 0;
  if (take > 0) {
    uint32_t lo = kNone, hi = max(code_max(x), kNone);
    int at_least = ncand, above = 0;           // scores >= lo, > hi
    // the best scores lie in the octaves below the largest: 4 of them (128 codes each) are tried first, then 32
    uint32_t reach = 512u;
    while (lo < hi && at_least != take) {
      uint32_t mid = (lo + hi + 1) / 2;
      if (reach != 0u) {
        mid = hi > lo + reach ? hi - reach : mid;
        reach = reach == 512u ? 4096u : 0u;
      }
      const int c = count_ge(x, mid);
      if (c >= take) {
        lo = mid;
        at_least = c;
        reach = 0u;
      } else {
        hi = mid - 1;
        above = c;
      }
    }
    t_code = lo;
    remaining = take - above;
    members = at_least - above;
    if (lo == kNone) ties = remaining;        // every number, and NaNs (key 0) in index order
  }
  // this lane's columns, round by round: bits of those that round above T, and to T
  __syncwarp();
  const __nv_bfloat162 t2 = as_pair(code_value(t_code) * 0x10001u);
  uint64_t gt[kRounds], eq[kRounds];
#pragma unroll
  for (int rd = 0; rd < kRounds; ++rd) {
    gt[rd] = eq[rd] = 0u;
    const int pair0 = (rd * 32 + lane) * kChunk;       // of this lane
    const int left = ncand - 2 * pair0;                // its candidates
    if (left > 0 && take > 0) {
#pragma unroll 8
      for (int i = 0; i < kChunk; ++i) {
        const float2 f = xs[slot(pair0 + i)];
        const __nv_bfloat162 v = as_pair(pack_bf16x2(f.x, f.y));
        uint32_t above_t, at_t;
        if (t_code == kNone) {
          above_t = __heq2_mask(v, v);
          at_t = ~above_t;
        } else {
          above_t = __hgt2_mask(v, t2);
          at_t = __heq2_mask(v, t2);
        }
        // a half of the mask is all ones or zeros: bits 0 and 31 tell
        gt[rd] |= static_cast<uint64_t>((above_t & 1u) | (above_t >> 31 << 1)) << (2 * i);
        eq[rd] |= static_cast<uint64_t>((at_t & 1u) | (at_t >> 31 << 1)) << (2 * i);
      }
      if (left < 64) {
        const uint64_t own = (1ull << left) - 1ull;
        gt[rd] &= own;
        eq[rd] &= own;
      }
    }
  }
  auto key_at = [&](int rd, int bit) {
    const float2 f = xs[slot((rd * 32 + lane) * kChunk + (bit >> 1))];
    return order_key(bit & 1 ? f.y : f.x);
  };
  if (t_code != kNone && remaining < members) {
    if (members <= 32) {
      // the members' full keys in a list, each ranked against all
      int mine_n = 0;
#pragma unroll
      for (int rd = 0; rd < kRounds; ++rd) mine_n += __popcll(eq[rd]);
      int at = mine_n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += v;
      }
      at -= mine_n;
#pragma unroll
      for (int rd = 0; rd < kRounds; ++rd)
        for (uint64_t m = eq[rd]; m; m &= m - 1) member_key[at++] = key_at(rd, __ffsll(m) - 1);
      __syncwarp();
      const uint32_t mine = lane < members ? member_key[lane] : 0u;
      int more = 0, same = 0;
      for (int i = 0; i < members; ++i) {
        const uint32_t other = member_key[i];
        more += other > mine ? 1 : 0;
        same += other == mine ? 1 : 0;
      }
      const bool is_it = lane < members && more < remaining && remaining <= more + same;
      const int src = __ffs(__ballot_sync(0xffffffffu, is_it)) - 1;
      thresh = __shfl_sync(0xffffffffu, mine, src);
      ties = remaining - __shfl_sync(0xffffffffu, more, src);
    } else {
      // many scores round to T: bisect their full keys
      int over = 0;
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t cand = thresh | (1u << bit);
        int c = 0;
#pragma unroll
        for (int rd = 0; rd < kRounds; ++rd)
          for (uint64_t m = eq[rd]; m; m &= m - 1) c += key_at(rd, __ffsll(m) - 1) >= cand ? 1 : 0;
        if (__reduce_add_sync(0xffffffffu, c) >= remaining) thresh = cand;
      }
#pragma unroll
      for (int rd = 0; rd < kRounds; ++rd)
        for (uint64_t m = eq[rd]; m; m &= m - 1) over += key_at(rd, __ffsll(m) - 1) > thresh ? 1 : 0;
      ties = remaining - __reduce_add_sync(0xffffffffu, over);
    }
  }
  int* out = idx_out + r * idx_stride;
  int kept = 0, equal = 0;
#pragma unroll
  for (int rd = 0; rd < kRounds; ++rd) {
    uint64_t sel = gt[rd], tie = 0u;
    if (__any_sync(0xffffffffu, eq[rd] != 0u)) {
      for (uint64_t m = eq[rd]; m; m &= m - 1) {
        const uint32_t key = key_at(rd, __ffsll(m) - 1);
        const uint64_t bit = m & (0ull - m);
        if (key > thresh) sel |= bit;
        if (key == thresh) tie |= bit;
      }
      // ties in index order: the first of those not yet taken by columns before this lane's
      const int nt = __popcll(tie);
      int before = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      const int all = __shfl_sync(0xffffffffu, before, 31);
      before += equal - nt;
      for (; tie != 0u && before < ties; tie &= tie - 1, ++before) sel |= tie & (0ull - tie);
      equal += all;
    }
    const int ns = __popcll(sel);
    int at = ns;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += v;
    }
    const int all = __shfl_sync(0xffffffffu, at, 31);
    at += kept - ns;
    for (; sel; sel &= sel - 1) out[at++] = (rd * 32 + lane) * 2 * kChunk + __ffsll(sel) - 1;
    kept += all;
  }
  if (n > 0) {
    if (lane == 0) out[kept] = n - 1;
    ++kept;
  }
  for (int t = kept + lane; t < idx_stride; t += 32) out[t] = -1;
  if (count_out && lane == 0) count_out[r] = kept;
}

}  // namespace topk_lens

cudaError_t launch_topk_lens(const float* scores, int rows, int ncols, const int* lens, int rows_per_len, int block,
                             int kb, int* idx_out, int idx_stride, int* count_out, uint32_t* status,
                             cudaStream_t st) {
  auto kernel = ncols <= 64 * 8 ? topk_lens::row_kernel<8>
                                : (ncols <= 64 * 32 ? topk_lens::row_kernel<32> : topk_lens::row_kernel<128>);
  return launch_dependent(kernel, dim3(rows), dim3(32), 0, st, scores, ncols, lens, rows_per_len, block, kb, idx_out,
                          idx_stride, count_out, status);
}

}  // namespace bsa
