// Queries and keys on their way from the projection to attention: every head's row is normalised
// by its root mean square, weighted, and rotated by its token's position, in one pass; the gradient
// of that; and the form that writes keys and values into a paged cache.
//
// One row x of d values, weight w, table row (cos, sin) of the token's position:
//   r = 1 / sqrt(mean(x^2) + eps),  y_i = x_i r w_i,
//   z_lo = y_lo cos - y_hi sin,  z_hi = y_hi cos + y_lo sin  for each pair (lo, hi) of the first
//   rot_dim columns: (i, i + rot_dim / 2), or (2 i, 2 i + 1) when interleaved; the rest z = y.
// With cos and sin times the weights of a column and of its partner (once per token), a row costs
// z_i = r (x_i wc_i + x_partner ws_i).  With several position axes pair i takes the position of
// the axis whose section holds i.
// Gradient, dy = the rotation's transpose of dz, g = dy w:
//   dx = r (g - x r^2 mean(g x)),   dw = sum over rows of dy x r.
//
// Bound by HBM: a row is read once and written once (the backward pass reads x and dz), all sums
// are fp32 in registers, the one rounding is the output's.  A lane holds 16 bytes of a row, so a
// bf16 row of 128 is 16 lanes and a warp-wide load is two whole rows; a warp takes kUnroll such
// loads of one token at once (every load is issued before the first is used) and reuses the
// token's table columns for all of them.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "common.cuh"

namespace attn {
namespace qkn {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;
constexpr int kMaxAxes = 4;

// Element strides of a [B][H][N][d] view (d contiguous).
struct View {
  long long b, h, n;
};

struct Params {
  const void* x[2];   // queries, keys
  void* out[2];       // forward: z; backward: dx
  const void* dz[2];  // backward
  const void* w[2];   // weights [d], or null: not normalised
  View xs[2], os[2], ds[2];
  const float* rope;  // [max_pos][rot]: cosines, then sines
  const int* pos;     // [axes][B][N] by the strides below
  long long pos_axis, pos_b;
  int end[kMaxAxes];  // first pair past each axis's section
  int axes, rot, max_pos;
  int B, N, H[2];
  float eps;
  float* dw;  // backward: partial weight gradients [blocks][2][d]
  // paged form: x[2..] are the values; tokens with a negative slot are left out
  const void* v;
  View vs;
  const int* slots;
  void* cache[2];
  int slots_total;
};

// 16 bytes of a row as fp32
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(dev::pack_bf16x2(f[0], f[1]), dev::pack_bf16x2(f[2], f[3]),
                      dev::pack_bf16x2(f[4], f[5]), dev::pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

// not the read-only path: the forward pass may run in place
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// The part of the row that lane `sub` of its row's lanes holds, and its partner's.
template <typename T, int D, bool kInter>
struct Lane {
  static constexpr int kV = Vec<T>::kN;
  static constexpr int kLanes = D / kV;      // lanes of a row
  static constexpr int kRows = 32 / kLanes;  // rows of a warp-wide load
  int sub, col, row;
  int partner;  // lane that holds the other half of this lane's pairs
  int sign;     // of the sine: -1 first half, +1 second half, 0 not rotated
  int pair;     // first pair
  __device__ __forceinline__ explicit Lane(int rot) {
    const int lane = threadIdx.x & 31;
    sub = lane % kLanes;
    row = lane / kLanes;
    col = sub * kV;
    partner = lane;
    sign = 0;
    pair = 0;
    if (col < rot) {
      if (kInter) {
        pair = col / 2;
        sign = 1;
      } else {
        const int half = rot / 2;
        sign = col < half ? -1 : 1;
        pair = col < half ? col : col - half;
        partner = col < half ? lane + half / kV : lane - half / kV;
      }
    }
  }
  // column of the pair partner of element e
  __device__ __forceinline__ int partner_col(int e, int rot) const {
    if (sign == 0) return col + e;
    if (kInter) return col + (e ^ 1);
    return col + e + (sign < 0 ? rot / 2 : -rot / 2);
  }
};

// cos and signed sin of this lane's columns for token (b, n).
template <typename T, int D, bool kInter>
__device__ __forceinline__ void load_angles(const Params& p, const Lane<T, D, kInter>& ln, int b,
                                            int n, float (&c)[Vec<T>::kN], float (&s)[Vec<T>::kN]) {
  constexpr int kV = Vec<T>::kN;
  constexpr int kPairs = kInter ? kV / 2 : kV;
#pragma unroll
  for (int e = 0; e < kV; ++e) c[e] = 1.f, s[e] = 0.f;
  if (ln.sign == 0) return;
  const int* pos = p.pos + b * p.pos_b + n;
  int at[kMaxAxes];
  bool in[kMaxAxes];
#pragma unroll
  for (int a = 0; a < kMaxAxes; ++a) {
    at[a] = a < p.axes ? __ldg(pos + a * p.pos_axis) : 0;
    in[a] = at[a] >= 0 && at[a] < p.max_pos;
  }
  float cc[kPairs], ss[kPairs];
  bool bad = false;
  auto axis_of = [&](int pair) {
    int a = 0;
#pragma unroll
    for (int i = 0; i < kMaxAxes - 1; ++i)
      if (i + 1 < p.axes && pair >= p.end[i]) a = i + 1;
    return a;
  };
  auto pick = [&](int a) { return a == 0 ? at[0] : a == 1 ? at[1] : a == 2 ? at[2] : at[3]; };
  auto okay = [&](int a) { return a == 0 ? in[0] : a == 1 ? in[1] : a == 2 ? in[2] : in[3]; };
  constexpr int kStep = kPairs >= 4 ? 4 : kPairs;
#pragma unroll
  for (int i = 0; i < kPairs; i += kStep) {
    const int a0 = axis_of(ln.pair + i), a1 = axis_of(ln.pair + i + kStep - 1);
    if (a0 == a1) {
      const float* row = p.rope + static_cast<size_t>(okay(a0) ? pick(a0) : 0) * p.rot + ln.pair + i;
      if (!okay(a0)) {
        bad = true;
#pragma unroll
        for (int e = 0; e < kStep; ++e) cc[i + e] = 1.f, ss[i + e] = 0.f;
      } else if constexpr (kStep == 4) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(row));
        const float4 y = __ldg(reinterpret_cast<const float4*>(row + p.rot / 2));
        cc[i] = x.x, cc[i + 1] = x.y, cc[i + 2] = x.z, cc[i + 3] = x.w;
        ss[i] = y.x, ss[i + 1] = y.y, ss[i + 2] = y.z, ss[i + 3] = y.w;
      } else {
        const float2 x = __ldg(reinterpret_cast<const float2*>(row));
        const float2 y = __ldg(reinterpret_cast<const float2*>(row + p.rot / 2));
        cc[i] = x.x, cc[i + 1] = x.y;
        ss[i] = y.x, ss[i + 1] = y.y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kStep; ++e) {
        const int a = axis_of(ln.pair + i + e);
        const float* row = p.rope + static_cast<size_t>(okay(a) ? pick(a) : 0) * p.rot + ln.pair + i + e;
        bad = bad || !okay(a);
        cc[i + e] = okay(a) ? __ldg(row) : 1.f;
        ss[i + e] = okay(a) ? __ldg(row + p.rot / 2) : 0.f;
      }
    }
  }
  // a position outside the table is not followed: its pairs are not rotated, and it is flagged
  if (bad) atomicExch(&g_device_error, ATTN_ERR_INVALID_ARG);
#pragma unroll
  for (int e = 0; e < kV; ++e) {
    c[e] = cc[kInter ? e / 2 : e];
    const float sn = ss[kInter ? e / 2 : e];
    s[e] = kInter ? ((e & 1) ? sn : -sn) : (ln.sign < 0 ? -sn : sn);
  }
}

// the values of each lane's pair partners
template <typename T, bool kInter>
__device__ __forceinline__ void partners(const uint4& raw, int lane, float (&f)[Vec<T>::kN]) {
  if (kInter) {
    float g[Vec<T>::kN];
    Vec<T>::unpack(raw, g);
#pragma unroll
    for (int e = 0; e < Vec<T>::kN; ++e) f[e] = g[e ^ 1];
  } else {
    uint4 u;
    u.x = __shfl_sync(0xffffffffu, raw.x, lane);
    u.y = __shfl_sync(0xffffffffu, raw.y, lane);
    u.z = __shfl_sync(0xffffffffu, raw.z, lane);
    u.w = __shfl_sync(0xffffffffu, raw.w, lane);
    Vec<T>::unpack(u, f);
  }
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A warp's item: kHeads heads of one token, all queries, all keys or all values.
template <typename T, int D, bool kInter, bool kPaged>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const Params p) {
  using L = Lane<T, D, kInter>;
  constexpr int kV = L::kV;
  constexpr int kHeads = kUnroll * L::kRows;
  const L ln(p.rot);
  const int cq = (p.H[0] + kHeads - 1) / kHeads, ck = (p.H[1] + kHeads - 1) / kHeads;
  const int chunks = cq + (kPaged ? 2 : 1) * ck;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const long long token = item / chunks;
  const int chunk = static_cast<int>(item % chunks);
  if (token >= static_cast<long long>(p.B) * p.N) return;
  const int b = static_cast<int>(token / p.N), n = static_cast<int>(token % p.N);
  const int kind = chunk < cq ? 0 : chunk < cq + ck ? 1 : 2;  // queries, keys, values
  const int side = kind == 0 ? 0 : 1;
  const int h0 = (chunk - (kind == 0 ? 0 : kind == 1 ? cq : cq + ck)) * kHeads + ln.row;
  const int H = p.H[side];
  long long slot = 0;
  if (kPaged) {
    slot = __ldg(p.slots + token);
    if (slot < 0) return;
    if (slot >= p.slots_total) {
      atomicExch(&g_device_error, ATTN_ERR_INVALID_ARG);
      return;
    }
  }
  const View& xs = (kPaged && kind == 2) ? p.vs : p.xs[side];
  const T* x = static_cast<const T*>((kPaged && kind == 2) ? p.v : p.x[side]) + b * xs.b + n * xs.n + ln.col;
  T* out;
  long long oh;
  if (kPaged && kind != 0) {
    out = static_cast<T*>(p.cache[kind - 1]) + slot * p.H[1] * D + ln.col;
    oh = D;
  } else {
    out = static_cast<T*>(p.out[side]) + b * p.os[side].b + n * p.os[side].n + ln.col;
    oh = p.os[side].h;
  }
  uint4 raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int h = h0 + u * L::kRows;
    raw[u] = h < H ? load16(x + h * xs.h) : make_uint4(0u, 0u, 0u, 0u);
  }
  if (kPaged && kind == 2) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * L::kRows;
      if (h < H) *reinterpret_cast<uint4*>(out + h * oh) = raw[u];
    }
    return;
  }
  const T* w = static_cast<const T*>(p.w[side]);
  float wc[kV], ws[kV];
  load_angles<T, D, kInter>(p, ln, b, n, wc, ws);
  if (w != nullptr) {
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      wc[e] *= static_cast<float>(w[ln.col + e]);
      ws[e] *= static_cast<float>(w[ln.partner_col(e, p.rot)]);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    float f[kV], g[kV];
    Vec<T>::unpack(raw[u], f);
    partners<T, kInter>(raw[u], ln.partner, g);
    float r = 1.f;
    if (w != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < kV; ++e) ss = fmaf(f[e], f[e], ss);
      r = rsqrtf(row_sum<L::kLanes>(ss) * (1.f / D) + p.eps);
    }
    // a column that is not rotated keeps its own value alone: no 0 x partner
#pragma unroll
    for (int e = 0; e < kV; ++e)
      f[e] = r * (ln.sign == 0 ? f[e] * wc[e] : fmaf(g[e], ws[e], f[e] * wc[e]));
    const int h = h0 + u * L::kRows;
    if (h < H) *reinterpret_cast<uint4*>(out + h * oh) = Vec<T>::pack(f);
  }
}

// Backward: persistent blocks; every warp takes items of the queries, then of the keys, and keeps
// the weight gradient of its columns in registers on the way; a block adds its warps' up in a fixed
// order and writes one partial row per side.
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_bwd_kernel(const Params p) {
  using L = Lane<T, D, kInter>;
  constexpr int kV = L::kV;
  constexpr int kHeads = kUnroll * L::kRows;
  __shared__ float red[kWarps * L::kRows][D];
  const L ln(p.rot);
  const int warp = threadIdx.x >> 5;
  const long long tokens = static_cast<long long>(p.B) * p.N;
  for (int side = 0; side < 2; ++side) {
    const int H = p.H[side];
    const int chunks = (H + kHeads - 1) / kHeads;
    const T* w = static_cast<const T*>(p.w[side]);
    float wt[kV], dw[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      wt[e] = w != nullptr ? static_cast<float>(w[ln.col + e]) : 1.f;
      dw[e] = 0.f;
    }
    for (long long item = static_cast<long long>(blockIdx.x) * kWarps + warp; item < tokens * chunks;
         item += static_cast<long long>(gridDim.x) * kWarps) {
      const long long token = item / chunks;
      const int h0 = static_cast<int>(item % chunks) * kHeads + ln.row;
      const int b = static_cast<int>(token / p.N), n = static_cast<int>(token % p.N);
      const View xs = p.xs[side], ds = p.ds[side], os = p.os[side];
      const T* x = static_cast<const T*>(p.x[side]) + b * xs.b + n * xs.n + ln.col;
      const T* dz = static_cast<const T*>(p.dz[side]) + b * ds.b + n * ds.n + ln.col;
      T* dx = static_cast<T*>(p.out[side]) + b * os.b + n * os.n + ln.col;
      uint4 rx[kUnroll], rz[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * L::kRows;
        rx[u] = rz[u] = make_uint4(0u, 0u, 0u, 0u);
        if (h < H) {
          rz[u] = load16(dz + h * ds.h);
          if (w != nullptr) rx[u] = load16(x + h * xs.h);
        }
      }
      float c[kV], s[kV];
      load_angles<T, D, kInter>(p, ln, b, n, c, s);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float dy[kV], g[kV];
        Vec<T>::unpack(rz[u], dy);
        partners<T, kInter>(rz[u], ln.partner, g);
        // the transpose turns the sine's sign
#pragma unroll
        for (int e = 0; e < kV; ++e)
          dy[e] = ln.sign == 0 ? dy[e] : fmaf(-g[e], s[e], dy[e] * c[e]);
        if (w != nullptr) {
          float f[kV];
          Vec<T>::unpack(rx[u], f);
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            ss = fmaf(f[e], f[e], ss);
            dot = fmaf(dy[e] * wt[e], f[e], dot);
          }
          ss = row_sum<L::kLanes>(ss);
          dot = row_sum<L::kLanes>(dot);
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          const float k = r * r * dot * (1.f / D);
          // rows past the last head are zeros and add nothing (unless eps is 0, hence the test)
          const bool live = h0 + u * L::kRows < H;
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            if (live) dw[e] = fmaf(dy[e] * r, f[e], dw[e]);
            dy[e] = r * fmaf(-f[e], k, dy[e] * wt[e]);
          }
        }
        const int h = h0 + u * L::kRows;
        if (h < H) *reinterpret_cast<uint4*>(dx + h * os.h) = Vec<T>::pack(dy);
      }
    }
    if (w != nullptr) {
#pragma unroll
      for (int e = 0; e < kV; ++e) red[warp * L::kRows + ln.row][ln.col + e] = dw[e];
      __syncthreads();
      for (int i = threadIdx.x; i < D; i += kThreads) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps * L::kRows; ++k) t += red[k][i];
        p.dw[(static_cast<size_t>(blockIdx.x) * 2 + side) * D + i] = t;
      }
      __syncthreads();
    }
  }
}

// Sum of the blocks' partial weight gradients, in a fixed order: a block of 32 x 32 threads takes
// 32 columns.  grid (d / 32, 2).
__global__ void __launch_bounds__(1024)
    qk_norm_dw_kernel(const float* __restrict__ part, int blocks, int d, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  float* out = blockIdx.y == 0 ? dwq : dwk;
  if (out == nullptr) return;
  const int i = threadIdx.x & 31, k = threadIdx.x >> 5, col = blockIdx.x * 32 + i;
  float t = 0.f;
  for (int r = k; r < blocks; r += 32) t += part[(static_cast<size_t>(r) * 2 + blockIdx.y) * d + col];
  red[k][i] = t;
  __syncthreads();
  if (k == 0) {
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) sum += red[r][i];
    out[col] = sum;
  }
}

}  // namespace qkn
}  // namespace attn
