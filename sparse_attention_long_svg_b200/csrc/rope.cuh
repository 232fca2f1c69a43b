// Per-head RMS norm of Q and K with the position rotation, written head-major
// (svg_qk_norm_rope), and its gradient (svg_qk_norm_rope_backward).
//
//   n = x r,  r = (mean x^2 + eps)^(-1/2);   y = R(pos) (w n)
//   u = R(pos)^T dy;  dw = sum over rows of u n;  g = w u;  dx = r (g - n mean(g n))
//
// R turns D/2 pairs of channels by the angles of one table row.  Both
// directions read every input once and write every output once, so HBM
// traffic bounds them.  A row is held by D/16 threads, 16 channels each: 8
// from the row's first half and the same 8 from its second half, so that
// either pairing (neighbours, or channel i with i + D/2) stays inside one
// thread and every access is 16 bytes.  A thread keeps its token's 8 cosines
// and sines while it walks over a chunk of the token's heads.
// Measured: forward 338 us for 32,760 tokens x 40 heads x D = 128 with V (2.03 GB,
// 6.0 TB/s); gradient 36 us + 5 us (dw) for 10,002 tokens, 32 / 8 heads, D = 64
// (175 MB, 4.9 TB/s; 8 heads to a chunk and 96 registers: 43 us).
#pragma once

#include "common.cuh"

namespace svg {

struct RopeArgs {
  // q, k, v: token-major [B, N, H, D] views (element strides), head-major rows [B*H, cap, D]
  const __nv_bfloat16 *x[3];
  int64_t xb[3], xn[3], xh[3];
  __nv_bfloat16 *y[3];
  const __nv_bfloat16 *dy[3];          // backward: gradients of y; dx has the views below
  __nv_bfloat16 *dx[3];
  int64_t db[3], dn[3], dh[3];
  int64_t cap[3];
  int heads[3];
  int chunks[3];                       // head chunks of each tensor
  const float *w[2];
  const float *cos, *sin;              // [P, D/2]; nullptr: no rotation
  const int32_t *start;                // [B] position of token 0; nullptr: 0
  float *partial;                      // backward: dw partial sums [q chunks, k chunks][gridDim.x][D]
  int B, N, P, hpt;                    // hpt: heads per chunk
  float eps;
};

constexpr int kRopeThreads = 128;       // 256: 6 us more of 338 (32,760 tokens x 40 heads, D = 128)

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<uint32_t *>(&b);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Turns the 16 channels (a: first half, b: second half) of one thread.
// INTER: neighbouring channels are a pair; else a[i] and b[i] are.
template <bool INTER>
__device__ __forceinline__ void rope_turn(float (&a)[8], float (&b)[8], const float (&cs)[8], const float (&sn)[8]) {
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
      a[2 * i] = a0 * cs[i] - a1 * sn[i];
      a[2 * i + 1] = a0 * sn[i] + a1 * cs[i];
      b[2 * i] = b0 * cs[4 + i] - b1 * sn[4 + i];
      b[2 * i + 1] = b0 * sn[4 + i] + b1 * cs[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i];
      a[i] = x * cs[i] - y * sn[i];
      b[i] = x * sn[i] + y * cs[i];
    }
  }
}

// This thread's 8 angles of table row `pos`.
template <int D, bool INTER>
__device__ __forceinline__ void rope_angles(const RopeArgs &p, int64_t pos, int c, float (&cs)[8], float (&sn)[8]) {
  const int64_t base = pos * (D / 2);
  const int i0 = INTER ? 4 * c : 8 * c, i1 = INTER ? D / 4 + 4 * c : 8 * c + 4;
  const float4 c0 = *reinterpret_cast<const float4 *>(p.cos + base + i0);
  const float4 c1 = *reinterpret_cast<const float4 *>(p.cos + base + i1);
  const float4 s0 = *reinterpret_cast<const float4 *>(p.sin + base + i0);
  const float4 s1 = *reinterpret_cast<const float4 *>(p.sin + base + i1);
  cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w;
  cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
  sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w;
  sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
}

// Whether a token's row of tensor t counts: a position that is not negative
// (padding), inside the table (for V as well: a cache row is whole or left
// alone) and, as `row`, inside the tensor's buffer.  Others than padding are recorded.
__device__ __forceinline__ bool rope_counts(const RopeArgs &p, int t, int64_t pos, int64_t row) {
  if (pos < 0) return false;
  if ((p.cos == nullptr || pos < p.P) && row < p.cap[t]) return true;
  record_error(SVG_ERR_DEVICE_CHECK, SVG_SITE_ROPE_RANGE);
  return false;
}

template <int D>
__device__ __forceinline__ void rope_weights(const float *w, int c, float (&wa)[8], float (&wb)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wa[i] = w ? w[8 * c + i] : 1.f;
    wb[i] = w ? w[D / 2 + 8 * c + i] : 1.f;
  }
}

// Sum over the D/16 threads of a row.
template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The chunk's tensor (0 q, 1 k, 2 v) and its first and last head.
__device__ __forceinline__ int rope_chunk(const RopeArgs &p, int chunk, int &h0, int &h1) {
  int t = 0;
  while (t < 2 && chunk >= p.chunks[t]) chunk -= p.chunks[t++];
  h0 = chunk * p.hpt;
  h1 = min(h0 + p.hpt, p.heads[t]);
  return t;
}

// One item = one token x one chunk of heads; U heads are in flight at a time.
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeArgs p) {
  constexpr int GT = D / 16;
  const int c = threadIdx.x % GT;
  const int64_t tokens = static_cast<int64_t>(p.B) * p.N;
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x) / GT;
  const int chunk = static_cast<int>(item / tokens);
  const bool live = chunk < p.chunks[0] + p.chunks[1] + p.chunks[2];   // dead groups still take part in shuffles
  const int64_t tok = item % tokens;
  const int b = static_cast<int>(tok / p.N), n = static_cast<int>(tok % p.N);
  int h0 = 0, h1 = 0;
  const int t = live ? rope_chunk(p, chunk, h0, h1) : 0;
  const int64_t pos = static_cast<int64_t>(p.start ? p.start[b] : 0) + n;
  const int64_t row = t == 0 ? n : pos;
  const bool ok = live && rope_counts(p, t, pos, row);
  float cs[8], sn[8], wa[8], wb[8];
  const bool turn = ok && t != 2 && p.cos != nullptr;
  if (turn) rope_angles<D, INTER>(p, pos, c, cs, sn);
  if (ok && t != 2) rope_weights<D>(p.w[t], c, wa, wb);
  const __nv_bfloat16 *x = p.x[t] + b * p.xb[t] + n * p.xn[t] + 8 * c;
  __nv_bfloat16 *y = p.y[t] + (static_cast<int64_t>(b) * p.heads[t] * p.cap[t] + row) * D + 8 * c;
  const bool store = ok || (live && t == 0);       // a padding row of Q becomes zero
  // every lane of a warp makes the same number of rounds, for the shuffles
  for (int i = 0; i < p.hpt; i += U) {
    uint4 va[U], vb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {      // without conditions, so that all are in flight
      const int h = max(min(h0 + i + u, h1 - 1), 0);
      va[u] = __ldcs(reinterpret_cast<const uint4 *>(x + h * p.xh[t]));
      vb[u] = __ldcs(reinterpret_cast<const uint4 *>(x + h * p.xh[t] + D / 2));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + i + u;
      float a[8], bb[8];
      unpack8(va[u], a);
      unpack8(vb[u], bb);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += a[j] * a[j] + bb[j] * bb[j];
      ss = row_sum<D>(ss);
      if (t != 2 && ok) {
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[j] *= r * wa[j];
          bb[j] *= r * wb[j];
        }
        if (turn) rope_turn<INTER>(a, bb, cs, sn);
        va[u] = pack8(a);
        vb[u] = pack8(bb);
      }
      if (store && h < h1) {
        __nv_bfloat16 *yr = y + h * p.cap[t] * D;
        const uint4 ya = ok ? va[u] : make_uint4(0, 0, 0, 0), yb = ok ? vb[u] : make_uint4(0, 0, 0, 0);
        if (U > 1) {                   // a large call: streaming, 15 us less of 338
          __stcs(reinterpret_cast<uint4 *>(yr), ya);
          __stcs(reinterpret_cast<uint4 *>(yr + D / 2), yb);
        } else {
          *reinterpret_cast<uint4 *>(yr) = ya;
          *reinterpret_cast<uint4 *>(yr + D / 2) = yb;
        }
      }
    }
  }
}

// grid (token tiles, head chunks): one CTA stays with one chunk, so that its
// threads sum dw of one tensor.  The next head's rows are on their way while a
// head is computed.  Sums run in fp32 over a thread's rows (at most 256: the
// host's choice of tiles) and a CTA's groups, and in fp64 over the CTAs.
constexpr int kRopeBackThreads = 128;

template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeBackThreads, 4) qk_norm_rope_backward_kernel(const RopeArgs p) {
  constexpr int GT = D / 16, GROUPS = kRopeBackThreads / GT;
  __shared__ float sums[GROUPS][D];
  const int c = threadIdx.x % GT, grp = threadIdx.x / GT;
  const int64_t tokens = static_cast<int64_t>(p.B) * p.N;
  int h0, h1;
  const int t = rope_chunk(p, blockIdx.y, h0, h1);
  float wa[8], wb[8], da[8], db[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) da[j] = db[j] = 0.f;
  if (t != 2) rope_weights<D>(p.w[t], c, wa, wb);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * GROUPS; base < tokens;
       base += static_cast<int64_t>(gridDim.x) * GROUPS) {
    const int64_t tok = base + grp;
    const bool live = tok < tokens;
    const int b = live ? static_cast<int>(tok / p.N) : 0, n = live ? static_cast<int>(tok % p.N) : 0;
    const int64_t pos = static_cast<int64_t>(p.start ? p.start[b] : 0) + n;
    const int64_t row = t == 0 ? n : pos;
    const bool ok = live && rope_counts(p, t, pos, row);
    const __nv_bfloat16 *x = t == 2 ? nullptr : p.x[t] + b * p.xb[t] + n * p.xn[t] + 8 * c;
    // rows that do not count are read all the same, at a row that exists
    const int64_t from = ok ? row : 0;
    const __nv_bfloat16 *dy = p.dy[t] + (static_cast<int64_t>(b) * p.heads[t] * p.cap[t] + from) * D + 8 * c;
    __nv_bfloat16 *dx = p.dx[t] + b * p.db[t] + n * p.dn[t] + 8 * c;
    uint4 ga, gb, xa, xb;
    auto load = [&](int next) {
      const int h = min(next, h1 - 1);
      ga = __ldcs(reinterpret_cast<const uint4 *>(dy + h * p.cap[t] * D));
      gb = __ldcs(reinterpret_cast<const uint4 *>(dy + h * p.cap[t] * D + D / 2));
      if (t != 2) {
        xa = __ldcs(reinterpret_cast<const uint4 *>(x + h * p.xh[t]));
        xb = __ldcs(reinterpret_cast<const uint4 *>(x + h * p.xh[t] + D / 2));
      }
    };
    load(h0);
    float cs[8], sn[8];
    const bool turn = ok && t != 2 && p.cos != nullptr;
    if (turn) {
      rope_angles<D, INTER>(p, pos, c, cs, sn);
#pragma unroll
      for (int j = 0; j < 8; ++j) sn[j] = -sn[j];          // the transposed rotation
    }
    for (int h = h0; h < h1; ++h) {
      if (t == 2) {                                         // one tensor per CTA: no divergence
        const uint4 va = ga, vb = gb;
        load(h + 1);
        if (live) {
          *reinterpret_cast<uint4 *>(dx + h * p.dh[t]) = ok ? va : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(dx + h * p.dh[t] + D / 2) = ok ? vb : make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      float u[8], v[8], a[8], bb[8];
      unpack8(ga, u);
      unpack8(gb, v);
      unpack8(xa, a);
      unpack8(xb, bb);
      load(h + 1);
      if (turn) rope_turn<INTER>(u, v, cs, sn);
      float ss = 0.f, gx = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss += a[j] * a[j] + bb[j] * bb[j];
        gx += u[j] * wa[j] * a[j] + v[j] * wb[j] * bb[j];
      }
      ss = row_sum<D>(ss);
      gx = row_sum<D>(gx);
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
      const float m = gx * r * (1.f / D);                   // mean of g n
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float na = a[j] * r, nb = bb[j] * r;
        if (ok) {
          da[j] += u[j] * na;
          db[j] += v[j] * nb;
        }
        u[j] = r * (u[j] * wa[j] - na * m);
        v[j] = r * (v[j] * wb[j] - nb * m);
      }
      if (live) {
        *reinterpret_cast<uint4 *>(dx + h * p.dh[t]) = ok ? pack8(u) : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(dx + h * p.dh[t] + D / 2) = ok ? pack8(v) : make_uint4(0, 0, 0, 0);
      }
    }
  }
  if (t == 2) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sums[grp][8 * c + j] = da[j];
    sums[grp][D / 2 + 8 * c + j] = db[j];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) s += sums[g][threadIdx.x];
    p.partial[(static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * D + threadIdx.x] = s;
  }
}

// dw[t] = sum of its partial rows: grid (D/8, 2), 128 row slices x 8 channels
// per CTA, added in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float *partial, int rows_q, int rows_k, float *dw_q,
                                                       float *dw_k) {
  __shared__ double part[128][8];
  float *dw = blockIdx.y == 0 ? dw_q : dw_k;
  if (dw == nullptr) return;
  const int rows = blockIdx.y == 0 ? rows_q : rows_k;
  const float *src = partial + (blockIdx.y == 0 ? 0 : static_cast<int64_t>(rows_q) * D);
  const int ch = threadIdx.x % 8, col = blockIdx.x * 8 + ch, slice = threadIdx.x / 8;
  double s = 0.0;
#pragma unroll 8
  for (int r = slice; r < rows; r += 128) s += static_cast<double>(src[static_cast<int64_t>(r) * D + col]);
  part[slice][ch] = s;
  __syncthreads();
  for (int n = 64; n > 0; n >>= 1) {
    if (slice < n) part[slice][ch] += part[slice + n][ch];
    __syncthreads();
  }
  if (slice == 0) dw[col] = static_cast<float>(part[0][ch]);
}

}  // namespace svg
