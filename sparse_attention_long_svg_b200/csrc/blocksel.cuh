// Mean keys of key blocks (svg_block_mean) and, for every query, the blocks
// with the largest score (svg_block_select).
//
//   mean[j] = sum of the block's keys / their number      (fp64 sum, one rounding)
//   score(n, j) = (sum over the group's heads of q[n]) . mean[j]
//
// The selection is an integer result, so it is the one that exact scores give,
// ties going to the lower block: scores are formed in fp32 with a known error
// bound e, and the candidates within 2e of the last place are compared again
// in fp64 (products of bf16 sums and fp32 means are exact there).  With t the
// approximate score in the last place, the exact one v satisfies |v - t| <= e,
// so a candidate above t + 2e is in, one below t - 2e is out.
#pragma once

#include "common.cuh"
#include "mma.cuh"
#include "rope.cuh"

namespace svg {

constexpr int kMaxBlocks = 4096;       // blocks of one sequence
constexpr int kMaxBlockTopk = 1024;

// Keys of a sequence: its entry of kv_len, kept inside the buffer.
__device__ __forceinline__ int seq_len(const int32_t *kv_len, int b, int Nk) {
  return kv_len ? min(max(kv_len[b], 0), Nk) : Nk;
}

// One CTA per (head, block): 256 threads = D/8 16-byte columns x row slots.
// HBM bound: reads the keys once.
template <int D>
__global__ void __launch_bounds__(256) block_mean_kernel(const __nv_bfloat16 *k, int Nk, int block, int nblk,
                                                         const int32_t *kv_len, int heads_per_seq, int fresh,
                                                         int per_head, float *mean) {
  constexpr int COLS = D / 8, SLOTS = 256 / COLS;
  __shared__ double sums[SLOTS][D];
  const int head = blockIdx.x / per_head;
  const int len = seq_len(kv_len, head / heads_per_seq, Nk);
  const int blk = blockIdx.x % per_head + (fresh > 0 ? max(0, len - fresh) / block : 0);
  if (blk >= nblk) return;
  const int rows = min(max(len - blk * block, 0), block);
  if (fresh > 0 && rows == 0) return;
  const int col = threadIdx.x % COLS, slot = threadIdx.x / COLS;
  const __nv_bfloat16 *src = k + (static_cast<int64_t>(head) * Nk + static_cast<int64_t>(blk) * block) * D + 8 * col;
  double acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0;
#pragma unroll 4
  for (int r = slot; r < rows; r += SLOTS) {
    float f[8];
    unpack8(__ldg(reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(r) * D)), f);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += static_cast<double>(f[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[slot][8 * col + i] = acc[i];
  __syncthreads();
  if (threadIdx.x < D) {
    double s = 0.0;
    for (int i = 0; i < SLOTS; ++i) s += sums[i][threadIdx.x];
    mean[(static_cast<int64_t>(head) * nblk + blk) * D + threadIdx.x] =
        rows > 0 ? static_cast<float>(s / static_cast<double>(rows)) : 0.f;
  }
}

struct SelectArgs {
  const __nv_bfloat16 *q;              // [BHk * G, Nq, D]
  const float *mean;                   // [BHk, nblk, D]
  const int32_t *kv_len;
  int32_t *sel;                        // [BHk, Nq, topk]
  float *scores;                       // prefill: per CTA [64][nblk]
  double *exact;                       // per warp [nblk]
  int BHk, G, heads_per_seq, Nq, Nk, nblk, block, topk, sink, local, causal;
};

// Order-preserving integers: larger value, larger key; NaN counts as -inf.
__device__ __forceinline__ uint32_t key32(float f) {
  if (f != f) f = -INFINITY;
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unkey32(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ uint64_t key64(double d) {
  if (d != d) d = -INFINITY;
  if (d == 0.0) d = 0.0;               // -0 and +0 are a tie
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(d));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

// What a query may select: blocks [0, may), of which [0, s1) and [l0, l1) are forced.
struct SelectRange {
  int may, s1, l0, l1;
  __device__ __forceinline__ bool forced(int j) const { return j < s1 || (j >= l0 && j < l1); }
  __device__ __forceinline__ int num_forced() const { return s1 + max(0, l1 - max(l0, s1)); }
};
__device__ __forceinline__ SelectRange select_range(const SelectArgs &a, int len, int n) {
  const int pos = len - a.Nq + n;
  const int seen = a.causal ? min(pos + 1, len) : len;
  SelectRange r;
  r.may = seen <= 0 ? 0 : (seen - 1) / a.block + 1;
  r.s1 = min(a.sink, r.may);
  r.l1 = pos < 0 ? 0 : min(pos / a.block + 1, r.may);
  r.l0 = max(0, r.l1 - a.local);
  return r;
}

// Exact score of block j: every lane returns it.
template <int D>
__device__ __forceinline__ double exact_score(const SelectArgs &a, const double (&qs)[D / 32], int head, int j) {
  const float *m = a.mean + (static_cast<int64_t>(head) * a.nblk + j) * D + lane_id() * (D / 32);
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) s += qs[i] * static_cast<double>(m[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// One warp writes one query's list.  s: approximate scores of the blocks
// [0, r.may); bound: their largest error; exact: scratch of nblk doubles.
// Block j belongs to lane j % 32, place j / 32.
template <int D, int VPL>
__device__ void select_row(const SelectArgs &a, const float *s, double *exact, float bound, int head, int n,
                           const SelectRange &r) {
  const int lane = lane_id();
  int32_t *out = a.sel + (static_cast<int64_t>(head) * a.Nq + n) * a.topk;
  const int places = (r.may + 31) / 32;
  const int forced = r.num_forced();
  int need = a.topk - forced;
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int j = i * 32 + lane;
    key[i] = (i < places && j < r.may && !r.forced(j)) ? key32(s[j]) : 0u;
  }
  // keep = key >= low (key 0 never is), and ties of the border resolved below
  uint32_t low = 1;
  bool border = false;
  float t = 0.f;
  if (r.may - forced > need) {
    uint32_t cut = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t trial = cut | (1u << bit);
      int c = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i < places) c += key[i] >= trial;
      c = __reduce_add_sync(0xffffffffu, c);
      if (c >= need) cut = trial;
      if (c == need) break;
    }
    // the last place's score, and who is near it
    uint32_t least = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i < places && key[i] >= cut && key[i] != 0) least = min(least, key[i]);
    low = need > 0 ? __reduce_min_sync(0xffffffffu, least) : 0xFFFFFFFFu;
    t = unkey32(low);
    int sure = 0, near = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i < places && key[i] != 0) {
        const float f = unkey32(key[i]);
        const bool above = f > t + 2.f * bound;
        sure += above;
        near += !above && !(f < t - 2.f * bound);
      }
    sure = __reduce_add_sync(0xffffffffu, sure);
    near = __reduce_add_sync(0xffffffffu, near);
    border = need > 0 && sure + near > need;
    need -= sure;
  }
  uint64_t cut64 = 0;
  int ties = 0;
  if (border) {
    double qs[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      qs[i] = 0.0;
      for (int g = 0; g < a.G; ++g)
        qs[i] += static_cast<double>(
            __bfloat162float(a.q[((static_cast<int64_t>(head) * a.G + g) * a.Nq + n) * D + lane * (D / 32) + i]));
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (i >= places) break;
      const float f = unkey32(key[i]);
      const bool near = key[i] != 0 && !(f > t + 2.f * bound) && !(f < t - 2.f * bound);
      uint32_t m = __ballot_sync(0xffffffffu, near);
      while (m) {
        const int l = __ffs(m) - 1;
        m &= m - 1;
        const double v = exact_score<D>(a, qs, head, i * 32 + l);
        if (lane == l) exact[i * 32 + l] = v;
      }
      if (near) key[i] = 1;                                        // marks a near one
      else if (key[i] != 0 && !(f > t + 2.f * bound)) key[i] = 0;  // out
    }
    // each lane reads back only what it wrote itself
    for (int bit = 63; bit >= 0; --bit) {
      const uint64_t trial = cut64 | (1ull << bit);
      int c = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i < places && key[i] == 1) c += key64(exact[i * 32 + lane]) >= trial;
      c = __reduce_add_sync(0xffffffffu, c);
      if (c >= need) cut64 = trial;
    }
    int above = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i < places && key[i] == 1) above += key64(exact[i * 32 + lane]) > cut64;
    ties = need - __reduce_add_sync(0xffffffffu, above);
  }
  int at = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (i >= places) break;
    const int j = i * 32 + lane;
    bool keep = j < r.may && r.forced(j);
    bool tie = false;
    if (border && key[i] == 1) {
      const uint64_t v = key64(exact[j]);
      keep = v > cut64;
      tie = v == cut64;
    } else if (key[i] != 0) {
      keep = border || key[i] >= low;
    }
    const uint32_t tied = __ballot_sync(0xffffffffu, tie);
    if (tie) keep = __popc(tied & ((1u << lane) - 1)) < ties;
    ties -= min(ties, __popc(tied));
    const uint32_t m = __ballot_sync(0xffffffffu, keep);
    if (keep) out[at + __popc(m & ((1u << lane) - 1))] = j;
    at += __popc(m);
  }
  for (int i = at + lane; i < a.topk; i += 32) out[i] = -1;
}

// Many queries: one CTA takes 64 queries of a key head and all their blocks.
// Scores run on the tensor cores with the summed queries and the means split
// into bf16 high and low parts: each low part's rounding and the omitted lo lo
// are at most 2^-16 of a product, the roundings of the fp32 sums (24 matrix
// steps) less than 2^-17, so the error is below 2^-14 |q| |mean| (norms of the
// head-wise absolute sum and of the block's mean).  The CTA's scores stay in
// its own scratch rows (read back from L2 by the same CTA).
constexpr int kSelTile = 64, kSelThreads = 128;
constexpr float kSelSplitError = 1.f / 16384.f;

template <int D>
constexpr int select_smem() {
  return 4 * kSelTile * D * 2;
}

__device__ __forceinline__ void split8(const float (&f)[8], uint4 &hi, uint4 &lo) {
  hi = pack8(f);
  float h[8], l[8];
  unpack8(hi, h);
#pragma unroll
  for (int i = 0; i < 8; ++i) l[i] = f[i] - h[i];
  lo = pack8(l);
}

template <int D, int VPL>
__global__ void __launch_bounds__(kSelThreads) block_select_kernel(const SelectArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float qn[kSelTile];       // |q| of every row
  __shared__ uint32_t mn;              // largest |mean|^2, as bits (values >= 0 order like integers)
  constexpr int TILE = kSelTile * D * 2, COLS = D / 8;
  const uint32_t base = smem_u32(smem);
  const uint32_t q_hi = base, q_lo = base + TILE, m_hi = base + 2 * TILE, m_lo = base + 3 * TILE;
  const int warp = warp_id(), lane = lane_id();
  const int qtiles = (a.Nq + kSelTile - 1) / kSelTile;
  const int64_t items = static_cast<int64_t>(qtiles) * a.BHk;
  float *scores = a.scores + static_cast<int64_t>(blockIdx.x) * kSelTile * a.nblk;
  double *exact = a.exact + (static_cast<int64_t>(blockIdx.x) * (kSelThreads / 32) + warp) * a.nblk;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int head = static_cast<int>(item % a.BHk);
    const int n0 = (qtiles - 1 - static_cast<int>(item / a.BHk)) * kSelTile;    // long causal rows first
    const int len = seq_len(a.kv_len, head / a.heads_per_seq, a.Nk);
    const int last = min(n0 + kSelTile, a.Nq) - 1;
    const int most = select_range(a, len, last).may;
    if (threadIdx.x == 0) mn = 0;
    __syncthreads();
    // queries: sum over heads, split
    for (int i = threadIdx.x; i < kSelTile * COLS; i += kSelThreads) {
      const int r = i / COLS, c = i % COLS;
      float f[8], ab = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = 0.f;
      if (n0 + r < a.Nq) {
        float w[8], z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = 0.f;
        for (int g = 0; g < a.G; ++g) {
          unpack8(__ldg(reinterpret_cast<const uint4 *>(
                      a.q + ((static_cast<int64_t>(head) * a.G + g) * a.Nq + n0 + r) * D + 8 * c)),
                  w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f[e] += w[e];
            z[e] += fabsf(w[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ab += z[e] * z[e];
      }
      uint4 hi, lo;
      split8(f, hi, lo);
      *reinterpret_cast<uint4 *>(smem + tile_at<D>(r, c)) = hi;
      *reinterpret_cast<uint4 *>(smem + TILE + tile_at<D>(r, c)) = lo;
#pragma unroll
      for (int o = COLS / 2; o > 0; o >>= 1) ab += __shfl_xor_sync(0xffffffffu, ab, o);
      if (c == 0) qn[r] = sqrtf(ab);
    }
    for (int j0 = 0; j0 < most; j0 += kSelTile) {
      for (int i = threadIdx.x; i < kSelTile * COLS; i += kSelThreads) {
        const int r = i / COLS, c = i % COLS;
        float f[8], nn = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
        if (j0 + r < most) {
          const float4 *src = reinterpret_cast<const float4 *>(
              a.mean + (static_cast<int64_t>(head) * a.nblk + j0 + r) * D + 8 * c);
          const float4 x = __ldg(src), y = __ldg(src + 1);
          f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
          f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) nn += f[e] * f[e];
        uint4 hi, lo;
        split8(f, hi, lo);
        *reinterpret_cast<uint4 *>(smem + 2 * TILE + tile_at<D>(r, c)) = hi;
        *reinterpret_cast<uint4 *>(smem + 3 * TILE + tile_at<D>(r, c)) = lo;
#pragma unroll
        for (int o = COLS / 2; o > 0; o >>= 1) nn += __shfl_xor_sync(0xffffffffu, nn, o);
        // a NaN or infinite mean makes every comparison an exact one
        if (c == 0) atomicMax(&mn, nn <= 3.4e38f ? __float_as_uint(nn) : 0x7F800000u);
      }
      __syncthreads();
      float acc[8][4];
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t ah[4], al[4];
        ldsm_x4(ldsm_a<D>(q_hi, 16 * warp, ks), ah);
        ldsm_x4(ldsm_a<D>(q_lo, 16 * warp, ks), al);
#pragma unroll
        for (int t = 0; t < 8; t += 2) {
          uint32_t bh[4], bl[4];
          ldsm_x4(ldsm_b<D>(m_hi, 8 * t, ks), bh);
          ldsm_x4(ldsm_b<D>(m_lo, 8 * t, ks), bl);
          mma_bf16(acc[t], al, bh[0], bh[1]);
          mma_bf16(acc[t + 1], al, bh[2], bh[3]);
          mma_bf16(acc[t], ah, bl[0], bl[1]);
          mma_bf16(acc[t + 1], ah, bl[2], bl[3]);
          mma_bf16(acc[t], ah, bh[0], bh[1]);
          mma_bf16(acc[t + 1], ah, bh[2], bh[3]);
        }
      }
      const int r0 = 16 * warp + frag_row();
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + (e >> 1) * 8, j = j0 + 8 * t + frag_col() + (e & 1);
          if (j < most) scores[static_cast<int64_t>(r) * a.nblk + j] = acc[t][e];
        }
      __syncthreads();
    }
    __syncthreads();
    const float mnorm = sqrtf(__uint_as_float(mn));
    for (int r = 16 * warp; r < 16 * warp + 16 && n0 + r < a.Nq; ++r) {
      float bound = kSelSplitError * qn[r] * mnorm;
      if (!(bound <= 3.4e38f)) bound = INFINITY;
      select_row<D, VPL>(a, scores + static_cast<int64_t>(r) * a.nblk, exact, bound, head, n0 + r,
                         select_range(a, len, n0 + r));
      __syncwarp();
    }
    __syncthreads();
  }
}

// Few queries: one CTA per (key head, query).  8 lanes (D = 64: 4) form one
// score in fp32; 16 products, two levels of sums: error below 2^-18 |q| |mean|.
// HBM bound: reads the means once.
constexpr int kSelDecodeThreads = 512;
constexpr float kSelDotError = 1.f / 262144.f;

template <int D, int VPL>
__global__ void __launch_bounds__(kSelDecodeThreads) block_select_decode_kernel(const SelectArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  double *exact = reinterpret_cast<double *>(smem);               // [nblk]
  float *scores = reinterpret_cast<float *>(exact + a.nblk);      // [nblk]
  __shared__ uint32_t mn;
  constexpr int GT = D / 16;
  const int head = blockIdx.x / a.Nq, n = blockIdx.x % a.Nq;
  const int len = seq_len(a.kv_len, head / a.heads_per_seq, a.Nk);
  const SelectRange r = select_range(a, len, n);
  const int c = threadIdx.x % GT;
  if (threadIdx.x == 0) mn = 0;
  float qs[16], qa = 0.f;
  {
    float z[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) qs[e] = z[e] = 0.f;
    for (int g = 0; g < a.G; ++g) {
      const uint4 *src = reinterpret_cast<const uint4 *>(
          a.q + ((static_cast<int64_t>(head) * a.G + g) * a.Nq + n) * D);
      float x[8], y[8];
      unpack8(__ldg(src + c), x);
      unpack8(__ldg(src + GT + c), y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        qs[e] += x[e];
        qs[8 + e] += y[e];
        z[e] += fabsf(x[e]);
        z[8 + e] += fabsf(y[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) qa += z[e] * z[e];
    qa = row_sum<D>(qa);
  }
  __syncthreads();
  uint32_t biggest = 0;
  const int rounds = (r.may + kSelDecodeThreads / GT - 1) / (kSelDecodeThreads / GT);
#pragma unroll 2
  for (int i = 0; i < rounds; ++i) {
    const int j = i * (kSelDecodeThreads / GT) + threadIdx.x / GT;
    float s = 0.f, nn = 0.f;
    if (j < r.may) {
      const float4 *src = reinterpret_cast<const float4 *>(a.mean + (static_cast<int64_t>(head) * a.nblk + j) * D);
      const float4 v[4] = {__ldg(src + 2 * c), __ldg(src + 2 * c + 1), __ldg(src + 2 * GT + 2 * c),
                           __ldg(src + 2 * GT + 2 * c + 1)};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s += v[e].x * qs[4 * e] + v[e].y * qs[4 * e + 1] + v[e].z * qs[4 * e + 2] + v[e].w * qs[4 * e + 3];
        nn += v[e].x * v[e].x + v[e].y * v[e].y + v[e].z * v[e].z + v[e].w * v[e].w;
      }
    }
    s = row_sum<D>(s);
    nn = row_sum<D>(nn);
    if (j < r.may && c == 0) scores[j] = s;
    biggest = max(biggest, nn <= 3.4e38f ? __float_as_uint(nn) : 0x7F800000u);
  }
  biggest = __reduce_max_sync(0xffffffffu, biggest);
  if (lane_id() == 0) atomicMax(&mn, biggest);
  __syncthreads();
  if (warp_id() == 0) {
    float bound = kSelDotError * sqrtf(qa) * sqrtf(__uint_as_float(mn));
    if (!(bound <= 3.4e38f)) bound = INFINITY;
    select_row<D, VPL>(a, scores, exact, bound, head, n, r);
  }
}

}  // namespace svg
