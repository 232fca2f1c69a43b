// Softmax attention of every query over the keys of its own list of key
// blocks (svg_block_attn) and its gradient (svg_block_attn_backward).
//
// The G = Hq/Hk query heads of a key head share the query's list, so the heads
// of neighbouring tokens form the rows of a matrix tile: floor(16/G) tokens with
// few queries (16-row tiles, here), floor(128/G) with many (tcgen05, in
// blockattn_tc.cuh).  A CTA marks its tokens' blocks in shared bit sets and walks
// over their union in ascending order; each row takes part in the blocks that
// its own token lists: others leave its maximum, sum and accumulator as they
// were (also where such a block holds infinities or NaN).  Here are the marking,
// the few-query kernel, and the gradient's work items and joins.
//
//   S = scale Q K^T over the visible keys;  m, l: running maximum and sum
//   O = sum exp(S - m) V / l;  lse = m + log l;  no visible key: O = 0, lse = -inf
// gradient, with P = exp(S - lse), delta = rowsum(dO O):
//   dS = P (dO V^T - delta);  dQ = scale dS K;  dK = scale dS^T Q;  dV = P^T dO
#pragma once

#include "blocksel.cuh"
#include "common.cuh"
#include "mma.cuh"

namespace svg {

constexpr int kBaTile = 64;            // keys per step
constexpr int kBaThreads = 128;
constexpr int kBaMaxGroup = 16;
constexpr int kBaMaxSplits = 64;

struct BlockAttnArgs {
  const __nv_bfloat16 *q, *k, *v;      // [BHk*G, Nq, D], [BHk, Nk, D]
  const int32_t *sel, *kv_len;         // [BHk, Nq, topk], [B] or nullptr
  __nv_bfloat16 *o;
  float *lse;                          // [BHk*G, Nq], may be nullptr
  float *part_o, *part_lse;            // splits: [splits][BHk*G*Nq][D], [splits][BHk*G*Nq] (log2 units)
  // backward
  const __nv_bfloat16 *dout, *out;
  const float *lse_in;
  float *delta;
  __nv_bfloat16 *dq, *dk, *dv;
  uint32_t *rev;                       // [BHk][nblk][ceil(Nq/32)] bit sets: who lists the block
  int32_t *item_first;                 // [BHk * key tiles + 1] first work item of a key tile
  int32_t *slot_first;                 // [BHk * key tiles] first slot of a tile with several items
  int32_t *items;                      // key tile of every work item
  float *part_kv;                      // [slot][2][64][D]
  int BHk, G, heads_per_seq, Nq, Nk, nblk, block, topk, causal, splits;
  int item_tokens, tile_tokens, k_stages;
  float scale, scale_log2;
  uint64_t wait_ns;
  int fault;                           // test hook: K and V (the gathered rows) are not loaded
};

// Keys the query n sees.
__device__ __forceinline__ int query_seen(const BlockAttnArgs &a, int len, int n) {
  return a.causal ? min(len - a.Nq + n + 1, len) : len;
}

// Bit sets of the blocks of `tokens` tokens from n0 on (word w of token t at
// bits[w * tokens + t], W words), their union as an ascending list; returns its
// length.  Ids outside the sequence and blocks without a visible key are passed
// over.  Called by all threads; uni: W words of scratch.
__device__ __forceinline__ int mark_blocks(const BlockAttnArgs &a, int head, int len, int n0, int tokens, int W,
                                           uint32_t *bits, uint32_t *uni, uint16_t *list, int *count) {
  constexpr int U = 8;                              // ids in flight per thread
  const int threads = blockDim.x, tid = threadIdx.x, lane = lane_id();
  for (int i = tid; i < tokens * W; i += threads) bits[i] = 0;
  const int32_t *sel = a.sel + (static_cast<int64_t>(head) * a.Nq + n0) * a.topk;
  const int ids = min(tokens, a.Nq - n0) * a.topk;
  // i / topk for i < 2^18 (tokens <= 128, topk <= 1024): the rounding of the
  // reciprocal adds less than 2^-14
  const uint32_t per = 0xFFFFFFFFu / a.topk + 1;
  __syncthreads();
  for (int i0 = tid; i0 < ids; i0 += U * threads) {
    int j[U];
#pragma unroll
    for (int u = 0; u < U; ++u) j[u] = __ldg(sel + min(i0 + u * threads, ids - 1));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * threads;
      if (i >= ids) break;
      const int tok = a.topk == 1 ? i : static_cast<int>(__umulhi(i, per));
      if (j[u] >= 0 && j[u] < a.nblk && static_cast<int64_t>(j[u]) * a.block < query_seen(a, len, n0 + tok))
        atomicOr(&bits[(j[u] >> 5) * tokens + tok], 1u << (j[u] & 31));
    }
  }
  __syncthreads();
  for (int w = warp_id(); w < W; w += threads / 32) {
    uint32_t u = 0;
    for (int t = lane; t < tokens; t += 32) u |= bits[w * tokens + t];
    u = __reduce_or_sync(0xffffffffu, u);
    if (lane == 0) uni[w] = u;
  }
  __syncthreads();
  if (warp_id() == 0) {
    int at = 0;
    for (int w0 = 0; w0 < W; w0 += 32) {
      const int w = w0 + lane;
      uint32_t u = w < W ? uni[w] : 0u;
      int pre = __popc(u);
      const int own = pre;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += x;
      }
      const int all = __shfl_sync(0xffffffffu, pre, 31);
      for (int i = 0; i < min(32, W - w0); ++i) {   // word by word, a lane to a bit
        const uint32_t x = __shfl_sync(0xffffffffu, u, i);
        const int p = at + __shfl_sync(0xffffffffu, pre - own, i);
        if ((x >> lane) & 1u) list[p + __popc(x & ((1u << lane) - 1))] = static_cast<uint16_t>((w0 + i) * 32 + lane);
      }
      at += all;
    }
    if (lane == 0) *count = at;
  }
  __syncthreads();
  return *count;
}

// Bytes of the bit sets, their union and its list.
__host__ __device__ constexpr size_t mark_bytes(int tokens, int nblk) {
  const size_t W = (nblk + 31) / 32;
  return (static_cast<size_t>(tokens) + 1) * W * 4 + static_cast<size_t>(nblk) * 2;
}

// Rows [key0, key0 + ROWS) of a [Nk, D] matrix to a shared tile by THREADS
// threads; rows from `len` on become zeros.
template <int D, int THREADS, int ROWS>
__device__ __forceinline__ void load_tile(uint32_t dst, const __nv_bfloat16 *src, int key0, int len, int tid) {
  constexpr int COLS = D / 8, STEP = THREADS / COLS;       // STEP rows at a time
  static_assert(STEP > 0 && ROWS % STEP == 0, "");
  const int r0 = tid / COLS, c = tid % COLS;
  const __nv_bfloat16 *from = src + static_cast<int64_t>(key0 + r0) * D + 8 * c;
  if (key0 + ROWS <= len) {
#pragma unroll
    for (int r = 0; r < ROWS; r += STEP) cp_async16(dst + tile_at<D>(r0 + r, c), from + r * D, 16);
  } else {
#pragma unroll
    for (int r = 0; r < ROWS; r += STEP) {
      const bool in = key0 + r0 + r < len;
      cp_async16(dst + tile_at<D>(r0 + r, c), in ? from + r * D : src, in ? 16u : 0u);
    }
  }
}

// A operand (16 rows x D channels) straight from global memory.
template <int D>
__device__ __forceinline__ void load_rows(uint32_t (&f)[D / 16][4], const __nv_bfloat16 *r0, const __nv_bfloat16 *r1) {
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const int c = 16 * ks + frag_col();
    f[ks][0] = r0 ? *reinterpret_cast<const uint32_t *>(r0 + c) : 0u;
    f[ks][1] = r1 ? *reinterpret_cast<const uint32_t *>(r1 + c) : 0u;
    f[ks][2] = r0 ? *reinterpret_cast<const uint32_t *>(r0 + c + 8) : 0u;
    f[ks][3] = r1 ? *reinterpret_cast<const uint32_t *>(r1 + c + 8) : 0u;
  }
}

// One row of a 16-row tile as this thread sees it.
struct BaRow {
  int64_t row;      // row of [BHk*G*Nq], -1: none
  int tok;          // token within the CTA's
  int seen;         // keys it sees
};
__device__ __forceinline__ BaRow ba_row(const BlockAttnArgs &a, int head, int len, int n0, int tok0, int r) {
  BaRow x;
  const int per = 16 / a.G;
  x.tok = tok0 + r / a.G;
  const int n = n0 + x.tok;
  const bool in = r < per * a.G && n < a.Nq;
  x.row = in ? (static_cast<int64_t>(head) * a.G + r % a.G) * a.Nq + n : -1;
  x.seen = in ? query_seen(a, len, n) : 0;
  if (!in) x.tok = tok0;
  return x;
}

// Shared memory: rows of K and V, then the list's length, bit sets, list.
template <int D>
__host__ __device__ constexpr size_t block_attn_smem(int rows, int tokens, int nblk) {
  return static_cast<size_t>(rows) * D * 2 + 16 + mark_bytes(tokens, nblk);
}

__device__ __forceinline__ float dot_rows(const __nv_bfloat16 *a, const __nv_bfloat16 *b, int D) {
  float s = 0.f;
  for (int c = 0; c < D; c += 8) {
    float x[8], y[8];
    unpack8(*reinterpret_cast<const uint4 *>(a + c), x);
    unpack8(*reinterpret_cast<const uint4 *>(b + c), y);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[e] * y[e];
  }
  return s;
}

// What the CTA's rows share, for the row that is computed again: tiles [u0, u1)
// of the union (key(u)), the row's bit set.
struct BaUnion {
  const uint16_t *list;
  const uint32_t *bits;
  int u0, u1, keys, shift, tokens;     // a block has 2^shift tiles of `keys` keys
  __device__ __forceinline__ int block_of(int u) const { return list[u >> shift]; }
  __device__ __forceinline__ int key(int u) const {
    return ((block_of(u) << shift) + (u & ((1 << shift) - 1))) * keys;
  }
  __device__ __forceinline__ bool listed(int tok, int u) const {
    const int j = block_of(u);
    return (bits[(j >> 5) * tokens + tok] >> (j & 31)) & 1u;
  }
};

// One row by one warp, from its own keys alone: two passes over the scores.
// Lane i ends with channels i * D/32 ... of the normalised output.
template <int D>
__device__ __noinline__ void row_again(const BaUnion &un, const __nv_bfloat16 *q, const __nv_bfloat16 *k,
                                       const __nv_bfloat16 *v, int tok, int seen, float sl2, float (&y)[D / 32],
                                       float &lse2) {
  constexpr int E = D / 32;
  const int lane = lane_id();
  float m = -INFINITY, l = 0.f;
  bool nan = false;
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    for (int u = un.u0; u < un.u1; ++u) {
      if (!un.listed(tok, u)) continue;
      const int key0 = un.key(u), end = min(seen - key0, un.keys);
      for (int j0 = 0; j0 < end; j0 += 32) {
        const bool in = j0 + lane < end;
        float s = -INFINITY;
        if (in) s = dot_rows(q, k + static_cast<int64_t>(key0 + j0 + lane) * D, D) * sl2;
        if (pass == 0) {
          m = fmaxf(m, s);
          nan = nan || s != s;
          continue;
        }
        const float p = in ? ex2_approx(s - m) : 0.f;
        l += p;
        for (int j = 0; j < min(32, end - j0); ++j) {
          const float pj = __shfl_sync(0xffffffffu, p, j);
          const __nv_bfloat16 *vr = v + static_cast<int64_t>(key0 + j0 + j) * D + lane * E;
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] += pj * __bfloat162float(vr[e]);
        }
      }
    }
    if (pass == 0) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (__any_sync(0xffffffffu, nan)) m = __int_as_float(0x7FC00000);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  // scores of minus infinity only: as without keys
  const float inv = m == -INFINITY ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = m == -INFINITY ? 0.f : y[e] * inv;
  lse2 = m == -INFINITY ? -INFINITY : m + log2f(l);
}

// Few queries (at most floor(16/G), single tokens among them): all warps hold
// the same 16 rows and take every fourth tile of 32 keys, each through its own
// three buffers, so that 128 KB and more are always on their way (HBM bound:
// each listed key is read once: 16 sequences x 8 heads x 32 blocks, 27 us, 4.9
// TB/s); the CTA joins the warps.  gridDim.y splits the
// union's tiles; a second kernel joins the splits.
constexpr int kFewKeys = 32, kFewStages = 3, kFewRows = 4 * kFewStages * 2 * kFewKeys;   // rows of shared memory

template <int D>
__global__ void __launch_bounds__(kBaThreads, 1) block_attn_few_kernel(const BlockAttnArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int KEYS = kFewKeys, STAGES = kFewStages, TILE = KEYS * D * 2, NT = D / 8, ST = KEYS / 8;
  const int per = 16 / a.G;                       // tokens of a warp
  const int tokens = per;
  const int ntiles = (a.Nq + tokens - 1) / tokens;
  const int head = blockIdx.x % a.BHk;
  const int n0 = (ntiles - 1 - static_cast<int>(blockIdx.x / a.BHk)) * tokens;   // long causal rows first
  const int W = (a.nblk + 31) / 32;
  const int warp = warp_id();
  int *count = reinterpret_cast<int *>(smem + kFewRows * D * 2);
  uint32_t *bits = reinterpret_cast<uint32_t *>(count + 4), *uni = bits + tokens * W;
  uint16_t *list = reinterpret_cast<uint16_t *>(uni + W);
  const int len = seq_len(a.kv_len, head / a.heads_per_seq, a.Nk);
  const int sub = a.block / KEYS;
  const BaRow x0 = ba_row(a, head, len, n0, 0, frag_row());
  const BaRow x1 = ba_row(a, head, len, n0, 0, frag_row() + 8);
  uint32_t qf[D / 16][4];
  load_rows<D>(qf, x0.row >= 0 ? a.q + x0.row * D : nullptr, x1.row >= 0 ? a.q + x1.row * D : nullptr);
  const int total = mark_blocks(a, head, len, n0, tokens, W, bits, uni, list, count) * sub;
  const int each = (total + a.splits - 1) / a.splits;
  const int u0 = min(static_cast<int>(blockIdx.y) * each, total), u1 = min(u0 + each, total);
  const __nv_bfloat16 *kh = a.k + static_cast<int64_t>(head) * a.Nk * D;
  const __nv_bfloat16 *vh = a.v + static_cast<int64_t>(head) * a.Nk * D;

  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

  const uint32_t base = smem_u32(smem);
  const int first = u0 + warp, step = 4;
  auto buffer = [&](int i) {
    return base + static_cast<uint32_t>(warp * STAGES + i % STAGES) * 2 * TILE;
  };
  auto key_of = [&](int u) { return static_cast<int>(list[u / sub]) * a.block + (u % sub) * KEYS; };
  auto fetch = [&](int i) {
    const int u = first + i * step;
    if (u < u1) {
      const int key0 = key_of(u);
      load_tile<D, 32, KEYS>(buffer(i), kh, key0, len, lane_id());
      load_tile<D, 32, KEYS>(buffer(i) + TILE, vh, key0, len, lane_id());
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  for (int i = 0; first + i * step < u1; ++i) {
    fetch(i + STAGES - 1);
    cp_async_wait<STAGES - 1>();
    __syncwarp();
    const int u = first + i * step;
    const int blk = list[u / sub], key0 = key_of(u);
    const bool on0 = x0.row >= 0 && ((bits[(blk >> 5) * tokens + x0.tok] >> (blk & 31)) & 1u) && key0 < x0.seen;
    const bool on1 = x1.row >= 0 && ((bits[(blk >> 5) * tokens + x1.tok] >> (blk & 31)) & 1u) && key0 < x1.seen;
    if (__any_sync(0xffffffffu, on0 || on1)) {
      const uint32_t kt = lane_b<D>(buffer(i)), vt = lane_a<D>(buffer(i) + TILE);
      float s[ST][4];
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int t = 0; t < ST; t += 2) {
          uint32_t b[4];
          ldsm_x4(piece<D>(kt, 8 * t, ks), b);
          mma_bf16(s[t], qf[ks], b[0], b[1]);
          mma_bf16(s[t + 1], qf[ks], b[2], b[3]);
        }
      const int end0 = on0 ? x0.seen - key0 : 0, end1 = on1 ? x1.seen - key0 : 0;
      if (!__all_sync(0xffffffffu, end0 >= KEYS && end1 >= KEYS)) {
#pragma unroll
        for (int t = 0; t < ST; ++t) {
          const int c = 8 * t + frag_col();
          s[t][0] = c < end0 ? s[t][0] : -INFINITY;
          s[t][1] = c + 1 < end0 ? s[t][1] : -INFINITY;
          s[t][2] = c < end1 ? s[t][2] : -INFINITY;
          s[t][3] = c + 1 < end1 ? s[t][3] : -INFINITY;
        }
      }
      float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
      for (int t = 0; t < ST; ++t) {
        t0 = fmaxf(t0, fmaxf(s[t][0], s[t][1]));
        t1 = fmaxf(t1, fmaxf(s[t][2], s[t][3]));
      }
      const float n0m = fmaxf(m0, quad_max(t0) * a.scale_log2), n1m = fmaxf(m1, quad_max(t1) * a.scale_log2);
      const float b0 = n0m == -INFINITY ? 0.f : n0m, b1 = n1m == -INFINITY ? 0.f : n1m;
      if (__any_sync(0xffffffffu, n0m != m0 || n1m != m1)) {      // a new maximum: rescale
        const float f0 = n0m != m0 ? ex2_approx(m0 - b0) : 1.f, f1 = n1m != m1 ? ex2_approx(m1 - b1) : 1.f;
        m0 = n0m;
        m1 = n1m;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          acc[t][0] *= f0;
          acc[t][1] *= f0;
          acc[t][2] *= f1;
          acc[t][3] *= f1;
        }
      }
      uint32_t p[ST / 2][4];
#pragma unroll
      for (int t = 0; t < ST; ++t) {
        const float p0 = ex2_approx(fmaf(s[t][0], a.scale_log2, -b0)), p1 = ex2_approx(fmaf(s[t][1], a.scale_log2, -b0));
        const float p2 = ex2_approx(fmaf(s[t][2], a.scale_log2, -b1)), p3 = ex2_approx(fmaf(s[t][3], a.scale_log2, -b1));
        l0 += p0 + p1;
        l1 += p2 + p3;
        // P as bf16 for the matrix product: 2^-8 relative to each weight; the sum keeps fp32
        p[t / 2][(t & 1) * 2] = pack_bf16(p0, p1);
        p[t / 2][(t & 1) * 2 + 1] = pack_bf16(p2, p3);
      }
      if (__all_sync(0xffffffffu, on0 && on1)) {
#pragma unroll
        for (int ks = 0; ks < KEYS / 16; ++ks)
#pragma unroll
          for (int t = 0; t < NT; t += 2) {
            uint32_t b[4];
            ldsm_x4_trans(piece<D>(vt, 16 * ks, t / 2), b);
            mma_bf16(acc[t], p[ks], b[0], b[1]);
            mma_bf16(acc[t + 1], p[ks], b[2], b[3]);
          }
      } else {
        // a row that does not list this block keeps its accumulator, whatever V holds
#pragma unroll
        for (int t = 0; t < NT; t += 4) {
          float c[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[j][e] = acc[t + j][e];
#pragma unroll
          for (int ks = 0; ks < KEYS / 16; ++ks)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              uint32_t b[4];
              ldsm_x4_trans(piece<D>(vt, 16 * ks, (t + j) / 2), b);
              mma_bf16(c[j], p[ks], b[0], b[1]);
              mma_bf16(c[j + 1], p[ks], b[2], b[3]);
            }
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[t + j][e] = (e < 2 ? on0 : on1) ? c[j][e] : acc[t + j][e];
        }
      }
    }
    __syncwarp();
  }
  cp_async_wait<0>();
  l0 = quad_sum(l0);
  l1 = quad_sum(l1);

  // join the four warps' sums: [warp][16 rows][D] and maxima / sums behind
  __syncthreads();
  float *so = reinterpret_cast<float *>(smem);
  float *sm = so + 4 * 16 * D, *sl = sm + 64;
  int *bad = reinterpret_cast<int *>(sl + 64);
  if (threadIdx.x < 16) bad[threadIdx.x] = 0;
  const int r0 = frag_row();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = 8 * t + frag_col();
    *reinterpret_cast<float2 *>(so + (warp * 16 + r0) * D + c) = make_float2(acc[t][0], acc[t][1]);
    *reinterpret_cast<float2 *>(so + (warp * 16 + r0 + 8) * D + c) = make_float2(acc[t][2], acc[t][3]);
  }
  if ((lane_id() & 3) == 0) {
    sm[warp * 16 + r0] = m0;
    sm[warp * 16 + r0 + 8] = m1;
    sl[warp * 16 + r0] = l0;
    sl[warp * 16 + r0 + 8] = l1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * D / 2; i += kBaThreads) {
    const int r = i / (D / 2), c = (i % (D / 2)) * 2;
    const BaRow x = ba_row(a, head, len, n0, 0, r);
    if (x.row < 0) continue;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = fmaxf(m, sm[w * 16 + r]);
    const float b = m == -INFINITY ? 0.f : m;
    float l = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = ex2_approx(sm[w * 16 + r] - b);
      const float2 v = *reinterpret_cast<const float2 *>(so + (w * 16 + r) * D + c);
      l += f * sl[w * 16 + r];
      // a warp without a visible key holds zeros
      y0 += f * v.x;
      y1 += f * v.y;
    }
    const bool none = m == -INFINITY && l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
    y0 *= inv;
    y1 *= inv;
    const float lse2 = none ? -INFINITY : m + log2f(l);
    if (!none && !(fabsf(y0) < INFINITY && fabsf(y1) < INFINITY)) bad[r] = 1;
    if (a.splits > 1) {
      const int64_t pr = static_cast<int64_t>(blockIdx.y) * a.BHk * a.G * a.Nq + x.row;
      *reinterpret_cast<float2 *>(a.part_o + pr * D + c) = make_float2(y0, y1);
      if (c == 0) a.part_lse[pr] = lse2;
    } else {
      *reinterpret_cast<uint32_t *>(a.o + x.row * D + c) = pack_bf16(y0, y1);
      if (c == 0 && a.lse) a.lse[x.row] = lse2 * 0.69314718055994531f;
    }
  }
  // Weights of zero do not stop an infinity or NaN: rows that are not finite
  // again, from their own keys (a later token's key in the same tile).
  __syncthreads();
  BaUnion un;
  un.list = list;
  un.bits = bits;
  un.u0 = u0;
  un.u1 = u1;
  un.keys = KEYS;
  un.shift = a.block == 64 ? 1 : 2;
  un.tokens = tokens;
  for (int r = warp; r < 16; r += 4) {
    if (!bad[r]) continue;
    const BaRow x = ba_row(a, head, len, n0, 0, r);
    float y[D / 32], z;
    row_again<D>(un, a.q + x.row * D, kh, vh, x.tok, x.seen, a.scale_log2, y, z);
    const int64_t pr = static_cast<int64_t>(blockIdx.y) * a.BHk * a.G * a.Nq + x.row;
#pragma unroll
    for (int e = 0; e < D / 32; e += 2) {
      if (a.splits > 1)
        *reinterpret_cast<float2 *>(a.part_o + pr * D + lane_id() * (D / 32) + e) = make_float2(y[e], y[e + 1]);
      else
        *reinterpret_cast<uint32_t *>(a.o + x.row * D + lane_id() * (D / 32) + e) = pack_bf16(y[e], y[e + 1]);
    }
    if (lane_id() == 0) {
      if (a.splits > 1)
        a.part_lse[pr] = z;
      else if (a.lse)
        a.lse[x.row] = z * 0.69314718055994531f;
    }
  }
}

// Joins the splits of a row: one warp per row.
template <int D>
__global__ void __launch_bounds__(128) block_attn_join_kernel(const BlockAttnArgs a) {
  constexpr int E = D / 32;
  const int64_t rows = static_cast<int64_t>(a.BHk) * a.G * a.Nq;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + warp_id();
  if (row >= rows) return;
  float m = -INFINITY;
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.part_lse[s * rows + row]);
  const float b = m == -INFINITY ? 0.f : m;
  float l = 0.f, y[E];
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const float z = a.part_lse[s * rows + row];
    const float f = z == -INFINITY ? 0.f : ex2_approx(z - b);
    l += f;
    const float *src = a.part_o + (s * rows + row) * D + lane_id() * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 v = *reinterpret_cast<const float2 *>(src + e);
      y[e] += f * v.x;
      y[e + 1] += f * v.y;
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t *>(a.o + row * D + lane_id() * E + e) = pack_bf16(y[e] * inv, y[e + 1] * inv);
  if (a.lse && lane_id() == 0) a.lse[row] = (l == 0.f ? -INFINITY : b + log2f(l)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ gradient
// Who lists a block: bit sets over the queries (order of the atomics is of no
// account).
__global__ void __launch_bounds__(256) block_attn_reverse_kernel(const BlockAttnArgs a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(a.BHk) * a.Nq * a.topk) return;
  const int64_t q = i / a.topk;
  const int head = static_cast<int>(q / a.Nq), n = static_cast<int>(q % a.Nq);
  const int len = seq_len(a.kv_len, head / a.heads_per_seq, a.Nk);
  const int j = a.sel[i];
  if (j < 0 || j >= a.nblk || static_cast<int64_t>(j) * a.block >= query_seen(a, len, n)) return;
  const int64_t WQ = (a.Nq + 31) / 32;
  atomicOr(a.rev + (static_cast<int64_t>(head) * a.nblk + j) * WQ + (n >> 5), 1u << (n & 31));
}

// Work items of every key tile: ceil(queries / item_tokens), at least one.  One
// warp counts a block's queries.
__global__ void __launch_bounds__(256) block_attn_count_kernel(const BlockAttnArgs a) {
  const int sub = a.block / kBaTile;
  const int64_t blk = static_cast<int64_t>(blockIdx.x) * 8 + warp_id();
  if (blk >= static_cast<int64_t>(a.BHk) * a.nblk) return;
  const int WQ = (a.Nq + 31) / 32;
  int c = 0;
  for (int w = lane_id(); w < WQ; w += 32) c += __popc(a.rev[blk * WQ + w]);
  c = __reduce_add_sync(0xffffffffu, c);
  if (static_cast<int>(lane_id()) < sub)
    a.item_first[blk * sub + lane_id()] = max(1, (c + a.item_tokens - 1) / a.item_tokens);
}

// Exclusive sums over the key tiles: items (in place) and slots (of tiles with
// several items), as the high and low half of one 64-bit sum; and the tile of
// every item.
__global__ void __launch_bounds__(1024) block_attn_items_kernel(const BlockAttnArgs a) {
  __shared__ unsigned long long warp_sum[32];
  const int tiles = a.BHk * a.nblk * (a.block / kBaTile);
  unsigned long long carry = 0;
  for (int t0 = 0; t0 < tiles; t0 += 1024) {
    const int t = t0 + threadIdx.x;
    const int v = t < tiles ? a.item_first[t] : 0;
    const unsigned long long own = (static_cast<unsigned long long>(v) << 32) | (v > 1 ? v : 0);
    unsigned long long x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (static_cast<int>(lane_id()) >= o) x += y;
    }
    if (lane_id() == 31) warp_sum[warp_id()] = x;
    __syncthreads();
    unsigned long long at = carry + x - own;
    for (int w = 0; w < 32; ++w) {
      if (w < static_cast<int>(warp_id())) at += warp_sum[w];
      carry += warp_sum[w];
    }
    if (t < tiles) {
      const int item = static_cast<int>(at >> 32);
      a.item_first[t] = item;
      a.slot_first[t] = static_cast<int>(at & 0xFFFFFFFFu);
      for (int i = 0; i < v; ++i) a.items[item + i] = t;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) a.item_first[tiles] = static_cast<int>(carry >> 32);
}

// Sum of the items of a key tile with several: one CTA per tile.
template <int D>
__global__ void __launch_bounds__(256) block_attn_dkv_join_kernel(const BlockAttnArgs a) {
  const int sub = a.block / kBaTile;
  const int tile = blockIdx.x;
  const int first = a.item_first[tile], last = a.item_first[tile + 1];
  if (last - first <= 1) return;
  const int64_t blk = tile / sub;
  const int head = static_cast<int>(blk / a.nblk);
  const int key0 = static_cast<int>(blk % a.nblk) * a.block + (tile % sub) * kBaTile;
  const float *slots = a.part_kv + static_cast<int64_t>(a.slot_first[tile]) * 2 * kBaTile * D;
  for (int i = threadIdx.x; i < kBaTile * D; i += 256) {          // pairs of channels, dK then dV
    const int e = 2 * i, which = e / (kBaTile * D), at = e % (kBaTile * D);
    float2 s = make_float2(0.f, 0.f);
    for (int it = 0; it < last - first; ++it) {
      const float2 v = *reinterpret_cast<const float2 *>(slots + static_cast<int64_t>(it) * 2 * kBaTile * D + e);
      s.x += v.x;
      s.y += v.y;
    }
    const int key = key0 + at / D;
    if (key < a.Nk)
      *reinterpret_cast<uint32_t *>((which ? a.dv : a.dk) + (static_cast<int64_t>(head) * a.Nk + key) * D + at % D) =
          pack_bf16(s.x, s.y);
  }
}

}  // namespace svg
