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
// are fp32 in registers, the one rounding is the output's.  What keeps a kernel of this kind from
// the memory's rate is its instructions, and the layout of a row over lanes follows from that:
//   - a lane holds 16 bytes of a row as two halves A and B: kH columns and their kH partners (i and
//     i + rot_dim / 2), or 2 kH adjacent columns when interleaved, so a pair never leaves its lane;
//   - a warp takes the same heads of every step-th token: weights stay in registers, the token's
//     table columns are loaded once for kUnroll row loads, addresses advance by additions;
//   - the kUnroll row sums are reduced together (each step of the exchange halves the values a lane
//     still carries), so r is computed once per row instead of once per lane and row;
//   - arithmetic is in pairs of fp32 values.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "common.cuh"

namespace attn {
namespace qkn {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;     // row loads of a warp's item, forward
constexpr int kUnrollBwd = 2;  // backward: of x and of dz
constexpr int kBlocks = 3;     // per SM, forward: 80 registers a thread
constexpr int kBlocksBwd = 2;  // per SM, backward
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
  // paged form: the values, and tokens with a negative slot are left out
  const void* v;
  View vs;
  const int* slots;
  void* cache[2];
  int slots_total;
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t z;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(dev::pack2(a.x, a.y)), "l"(dev::pack2(b.x, b.y)));
  return dev::unpack2(z);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  return dev::unpack2(dev::fma2(dev::pack2(a.x, a.y), dev::pack2(b.x, b.y), dev::pack2(c.x, c.y)));
}

// One half of a lane's 16 bytes as fp32 pairs
template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
  static constexpr int kH = 4, kP = 2;  // columns, pairs of columns
  static __device__ __forceinline__ void unpack(uint32_t a, uint32_t b, float2 (&f)[2]) {
    f[0] = make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
    f[1] = make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
  }
  static __device__ __forceinline__ uint2 pack(const float2 (&f)[2]) {
    return make_uint2(dev::pack_bf16x2(f[0].x, f[0].y), dev::pack_bf16x2(f[1].x, f[1].y));
  }
};
template <>
struct Half<float> {
  static constexpr int kH = 2, kP = 1;
  static __device__ __forceinline__ void unpack(uint32_t a, uint32_t b, float2 (&f)[1]) {
    f[0] = make_float2(__uint_as_float(a), __uint_as_float(b));
  }
  static __device__ __forceinline__ uint2 pack(const float2 (&f)[1]) {
    return make_uint2(__float_as_uint(f[0].x), __float_as_uint(f[0].y));
  }
};

// A lane's place in its row.  kFull: rot_dim == d.
template <typename T, int D, bool kInter, bool kFull>
struct Lane {
  static constexpr int kH = Half<T>::kH, kP = Half<T>::kP;
  static constexpr int kLanes = D / (2 * kH);  // lanes of a row
  static constexpr int kRows = 32 / kLanes;    // rows of a warp-wide load
  int row, sub;
  int col, gap;  // first column of A, columns from A to B
  bool turned;   // the lane's columns are rotated
  __device__ __forceinline__ explicit Lane(int rot) {
    const int lane = threadIdx.x & 31;
    row = lane / kLanes;
    sub = lane % kLanes;
    turned = kFull || sub < rot / (2 * kH);
    col = (!kInter && turned ? kH : 2 * kH) * sub;
    gap = kInter || !turned ? kH : kFull ? D / 2 : rot / 2;
  }
  __device__ __forceinline__ int pair() const { return kH * sub; }
  __device__ __forceinline__ uint4 load(const T* p) const {
    uint4 r;
    // not the read-only path: the forward pass may run in place
    if constexpr (kInter) {
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    } else {
      asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
      asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                   : "=r"(r.z), "=r"(r.w) : "l"(p + gap) : "memory");
    }
    return r;
  }
  __device__ __forceinline__ void store(T* p, uint2 a, uint2 b) const {
    if constexpr (kInter) {
      *reinterpret_cast<uint4*>(p) = make_uint4(a.x, a.y, b.x, b.y);
    } else {
      *reinterpret_cast<uint2*>(p) = a;
      *reinterpret_cast<uint2*>(p + gap) = b;
    }
  }
  // weights of the lane's columns (1 without)
  __device__ __forceinline__ void weights(const T* w, float2 (&a)[kP], float2 (&b)[kP]) const {
#pragma unroll
    for (int e = 0; e < kP; ++e) {
      a[e] = b[e] = make_float2(1.f, 1.f);
      if (w != nullptr) {
        const T* wa = w + col + 2 * e;
        a[e] = make_float2(static_cast<float>(wa[0]), static_cast<float>(wa[1]));
        b[e] = make_float2(static_cast<float>(wa[gap]), static_cast<float>(wa[gap + 1]));
      }
    }
  }
};

// A token's positions, one per axis (kMulti) or the only one.
template <bool kMulti>
struct Pos {
  int at[kMulti ? kMaxAxes : 1];
  __device__ __forceinline__ void load(const Params& p, int b, int n) {
    if (p.rot == 0) {
      at[0] = 0;
      return;
    }
    const int* pos = p.pos + b * p.pos_b + n;
#pragma unroll
    for (int a = 0; a < (kMulti ? kMaxAxes : 1); ++a)
      at[a] = (!kMulti || a < p.axes) ? __ldg(pos + a * p.pos_axis) : 0;
  }
  __device__ __forceinline__ int pick(int a) const {
    if constexpr (kMulti)
      return a == 0 ? at[0] : a == 1 ? at[1] : a == 2 ? at[2] : at[3];
    else
      return at[0];
  }
};

__device__ __forceinline__ int axis_of(const Params& p, int pair) {
  int a = 0;
#pragma unroll
  for (int i = 0; i < kMaxAxes - 1; ++i)
    if (i + 1 < p.axes && pair >= p.end[i]) a = i + 1;
  return a;
}

// cos and sin of this lane's kH pairs.  A position outside the table is not followed: its pairs are
// not rotated, and it is flagged.
template <typename T, int D, bool kInter, bool kFull, bool kMulti>
struct Angles {
  using L = Lane<T, D, kInter, kFull>;
  static constexpr int kH = L::kH, kP = L::kP;
  float c[kH], s[kH];
  __device__ __forceinline__ void load(const Params& p, const L& ln, const Pos<kMulti>& pos) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kH; ++i) c[i] = 1.f, s[i] = 0.f;
    if (ln.turned) {
      const int rot = kFull ? D : p.rot;
      const int a0 = kMulti ? axis_of(p, ln.pair()) : 0;
      if (!kMulti || a0 == axis_of(p, ln.pair() + kH - 1)) {
        const int at = pos.pick(a0);
        bad = at < 0 || at >= p.max_pos;
        if (!bad) {
          const float* row = p.rope + static_cast<size_t>(at) * rot + ln.pair();
          if constexpr (kH == 4) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(row));
            const float4 y = __ldg(reinterpret_cast<const float4*>(row + rot / 2));
            c[0] = x.x, c[1] = x.y, c[2] = x.z, c[3] = x.w;
            s[0] = y.x, s[1] = y.y, s[2] = y.z, s[3] = y.w;
          } else {
            const float2 x = __ldg(reinterpret_cast<const float2*>(row));
            const float2 y = __ldg(reinterpret_cast<const float2*>(row + rot / 2));
            c[0] = x.x, c[1] = x.y;
            s[0] = y.x, s[1] = y.y;
          }
        }
      } else {  // the border of two sections
#pragma unroll
        for (int e = 0; e < kH; ++e) {
          const int at = pos.pick(axis_of(p, ln.pair() + e));
          if (at >= 0 && at < p.max_pos) {
            const float* row = p.rope + static_cast<size_t>(at) * rot + ln.pair() + e;
            c[e] = __ldg(row);
            s[e] = __ldg(row + rot / 2);
          } else {
            bad = true;
          }
        }
      }
    }
    if (bad) atomicExch(&g_device_error, ATTN_ERR_INVALID_ARG);
  }
  // (cos, cos) and (-sin, sin) of the columns that pair of columns e of half A / B stands for
  __device__ __forceinline__ float2 cosine(bool second, int e) const {
    if constexpr (kInter) {
      const float x = second ? c[kP + e] : c[e];
      return make_float2(x, x);
    } else {
      return make_float2(c[2 * e], c[2 * e + 1]);
    }
  }
  __device__ __forceinline__ float2 sine(bool second, int e) const {
    if constexpr (kInter) {
      const float x = second ? s[kP + e] : s[e];
      return make_float2(-x, x);
    } else {
      return second ? make_float2(s[2 * e], s[2 * e + 1]) : make_float2(-s[2 * e], -s[2 * e + 1]);
    }
  }
};

__device__ __forceinline__ float2 swap2(float2 x) { return make_float2(x.y, x.x); }

// f = f cf + partner sf for both halves (partner: the other half, or the neighbour when interleaved).
// A lane that is not rotated keeps f cf alone: no 0 x partner.
template <typename L, bool kInter, bool kFull>
__device__ __forceinline__ void turn(const L& ln, float2 (&a)[L::kP], float2 (&b)[L::kP],
                                     const float2 (&ca)[L::kP], const float2 (&sa)[L::kP],
                                     const float2 (&cb)[L::kP], const float2 (&sb)[L::kP]) {
#pragma unroll
  for (int e = 0; e < L::kP; ++e) {
    const float2 pa = kInter ? swap2(a[e]) : b[e], pb = kInter ? swap2(b[e]) : a[e];
    const float2 ya = mul2(a[e], ca[e]), yb = mul2(b[e], cb[e]);
    const float2 za = fma2(pa, sa[e], ya), zb = fma2(pb, sb[e], yb);
    a[e] = kFull || ln.turned ? za : ya;
    b[e] = kFull || ln.turned ? zb : yb;
  }
}

// Sums of four values over the kLanes lanes of a row; the lane ends with the sum of value
// 2 * (its bit kLanes / 2) + (its bit kLanes / 4).
template <int kLanes>
__device__ __forceinline__ float sum4(float v0, float v1, float v2, float v3) {
  const int lane = threadIdx.x & 31;
  const bool hi = lane & (kLanes / 2), odd = lane & (kLanes / 4);
  const float a = (hi ? v2 : v0) + __shfl_xor_sync(0xffffffffu, hi ? v0 : v2, kLanes / 2);
  const float b = (hi ? v3 : v1) + __shfl_xor_sync(0xffffffffu, hi ? v1 : v3, kLanes / 2);
  float x = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, kLanes / 4);
#pragma unroll
  for (int o = kLanes / 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// the value that sum4's lane for value i holds
template <int kLanes>
__device__ __forceinline__ float from4(float x, int i) {
  const int base = threadIdx.x & (32 - kLanes);
  return __shfl_sync(0xffffffffu, x, base + (i >> 1) * (kLanes / 2) + (i & 1) * (kLanes / 4));
}

// Which heads and tokens a warp takes: the same heads (queries, keys or values) of every step-th
// token, with the token's place (b, n) and its offsets kept up by additions.
struct Walk {
  int kind, h0, left;    // left: tokens from the current one to the end
  int step, step_b, step_n;
  int b, n;
  __device__ __forceinline__ Walk(const Params& p, int heads, bool paged) {
    const int cq = (p.H[0] + heads - 1) / heads, ck = (p.H[1] + heads - 1) / heads;
    const int chunks = cq + (paged ? 2 : 1) * ck;
    const int warps = gridDim.x * kWarps, w = blockIdx.x * kWarps + (threadIdx.x >> 5);
    step = warps / chunks;  // the launch has chunks warps at least
    const int token = w / chunks, chunk = w % chunks;
    left = token < step ? p.B * p.N - token : 0;
    kind = chunk < cq ? 0 : chunk < cq + ck ? 1 : 2;
    h0 = (chunk - (kind == 0 ? 0 : kind == 1 ? cq : cq + ck)) * heads;
    b = token / p.N;
    n = token % p.N;
    step_b = step / p.N;
    step_n = step % p.N;
  }
  __device__ __forceinline__ bool live() const { return left > 0; }
  __device__ __forceinline__ void next(const Params& p) {
    left -= step;
    b += step_b;
    n += step_n;
    if (n >= p.N) {
      n -= p.N;
      ++b;
    }
  }
};

// Strides that every token needs again: kept in shared memory and read there each time, so that they
// do not hold registers through the loop (the loops below run at 80 registers, three blocks per SM).
struct Strides {
  long long b, n;
  __device__ __forceinline__ void set(const View& v) volatile { b = v.b, n = v.n; }
  __device__ __forceinline__ long long at(int ib, int in) const volatile { return ib * b + in * n; }
};

// Forward.
template <typename T, int D, bool kInter, bool kFull, bool kMulti, bool kPaged>
__global__ void __launch_bounds__(kThreads, kBlocks) qk_norm_rope_kernel(const Params p) {
  using L = Lane<T, D, kInter, kFull>;
  constexpr int kP = L::kP;
  __shared__ volatile Strides st[3][2];  // of a kind's input and output
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) st[i][0].set(p.xs[i]), st[i][1].set(p.os[i]);
    st[2][0].set(p.vs);
  }
  __syncthreads();
  const L ln(p.rot);
  Walk wk(p, kUnroll * L::kRows, kPaged);
  if (!wk.live()) return;
  const int side = wk.kind == 0 ? 0 : 1;
  const bool copy = kPaged && wk.kind == 2;      // values: as they are
  const bool to_cache = kPaged && wk.kind != 0;
  const int h0 = wk.h0 + ln.row, H = p.H[side];
  const View& xs = copy ? p.vs : p.xs[side];
  const View& os = p.os[side];
  const T* x0 = static_cast<const T*>(copy ? p.v : p.x[side]) + h0 * xs.h + ln.col;
  T* out0 = to_cache ? static_cast<T*>(p.cache[wk.kind - 1]) + h0 * D + ln.col
                     : static_cast<T*>(p.out[side]) + h0 * os.h + ln.col;
  const long long xh = xs.h * L::kRows, oh = (to_cache ? D : os.h) * L::kRows;
  const T* w = copy ? nullptr : static_cast<const T*>(p.w[side]);
  float2 wa[kP], wb[kP];
  ln.weights(w, wa, wb);
  // the cache slot of the walk's token (below 0: left out)
  auto slot_of = [&](const Walk& k) -> int {
    if (!kPaged) return 0;
    const int s = __ldg(p.slots + k.n);
    if (s < p.slots_total) return s;
    atomicExch(&g_device_error, ATTN_ERR_INVALID_ARG);
    return -1;
  };
  Pos<kMulti> pos;
  if (!copy) pos.load(p, wk.b, wk.n);
  int slot = slot_of(wk);
  while (true) {
    const int b = wk.b, n = wk.n, cur = slot;
    const Pos<kMulti> cur_pos = pos;
    wk.next(p);
    const bool on = !kPaged || cur >= 0;
    uint4 raw[kUnroll];
    if (on) {
      const T* x = x0 + st[wk.kind][0].at(b, n);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        raw[u] = h0 + u * L::kRows < H ? ln.load(x + u * xh) : make_uint4(0u, 0u, 0u, 0u);
    }
    // the next token's position and slot are on their way meanwhile
    if (wk.live()) {
      if (!copy) pos.load(p, wk.b, wk.n);
      slot = slot_of(wk);
    }
    if (on) {
      T* out = to_cache ? out0 + static_cast<long long>(cur) * p.H[1] * D : out0 + st[wk.kind][1].at(b, n);
      if (copy) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (h0 + u * L::kRows < H)
            ln.store(out + u * oh, make_uint2(raw[u].x, raw[u].y), make_uint2(raw[u].z, raw[u].w));
      } else {
        Angles<T, D, kInter, kFull, kMulti> ang;
        ang.load(p, ln, cur_pos);
        // angle times weight: the column's own, and the partner's
        float2 ca[kP], sa[kP], cb[kP], sb[kP];
#pragma unroll
        for (int e = 0; e < kP; ++e) {
          ca[e] = mul2(wa[e], ang.cosine(false, e));
          cb[e] = mul2(wb[e], ang.cosine(true, e));
          sa[e] = mul2(kInter ? swap2(wa[e]) : wb[e], ang.sine(false, e));
          sb[e] = mul2(kInter ? swap2(wb[e]) : wa[e], ang.sine(true, e));
        }
        float r4 = 1.f;
        if (w != nullptr) {
          float ss[kUnroll];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            float2 fa[kP], fb[kP];
            Half<T>::unpack(raw[u].x, raw[u].y, fa);
            Half<T>::unpack(raw[u].z, raw[u].w, fb);
            float2 t = mul2(fa[0], fa[0]);
#pragma unroll
            for (int e = 1; e < kP; ++e) t = fma2(fa[e], fa[e], t);
#pragma unroll
            for (int e = 0; e < kP; ++e) t = fma2(fb[e], fb[e], t);
            ss[u] = t.x + t.y;
          }
          r4 = rsqrtf(sum4<L::kLanes>(ss[0], ss[1], ss[2], ss[3]) * (1.f / D) + p.eps);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const float r = from4<L::kLanes>(r4, u);
          const float2 rr = make_float2(r, r);
          float2 fa[kP], fb[kP];
          Half<T>::unpack(raw[u].x, raw[u].y, fa);
          Half<T>::unpack(raw[u].z, raw[u].w, fb);
          turn<L, kInter, kFull>(ln, fa, fb, ca, sa, cb, sb);
#pragma unroll
          for (int e = 0; e < kP; ++e) fa[e] = mul2(fa[e], rr), fb[e] = mul2(fb[e], rr);
          if (h0 + u * L::kRows < H) ln.store(out + u * oh, Half<T>::pack(fa), Half<T>::pack(fb));
        }
      }
    }
    if (!wk.live()) break;
  }
}

// Backward, walked the same way, with the next token's rows on their way while the current one's are
// worked on; a warp keeps the weight gradient of its columns in registers, and a block adds its
// warps' up in a fixed order into one partial row per side.
template <typename T, int D, bool kInter, bool kFull, bool kMulti>
__global__ void __launch_bounds__(kThreads, kBlocksBwd) qk_norm_rope_bwd_kernel(const Params p) {
  using L = Lane<T, D, kInter, kFull>;
  constexpr int kP = L::kP;
  __shared__ float red[kWarps * L::kRows][D];
  __shared__ int red_side[kWarps];
  __shared__ volatile Strides st[2][3];  // of a side's x, dz and dx
  if (threadIdx.x < 2) {
    st[threadIdx.x][0].set(p.xs[threadIdx.x]);
    st[threadIdx.x][1].set(p.ds[threadIdx.x]);
    st[threadIdx.x][2].set(p.os[threadIdx.x]);
  }
  __syncthreads();
  const L ln(p.rot);
  Walk wk(p, kUnrollBwd * L::kRows, false);
  const int warp = threadIdx.x >> 5, side = wk.kind;
  const int h0 = wk.h0 + ln.row, H = p.H[side];
  const T* x0 = static_cast<const T*>(p.x[side]) + ln.col;
  const T* dz0 = static_cast<const T*>(p.dz[side]) + ln.col;
  T* dx0 = static_cast<T*>(p.out[side]) + ln.col;
  // a row past the last head is loaded as the last head's and neither written nor counted
  long long xh[kUnrollBwd], dh[kUnrollBwd], oh[kUnrollBwd];
  bool live[kUnrollBwd];
#pragma unroll
  for (int u = 0; u < kUnrollBwd; ++u) {
    const int h = min(h0 + u * L::kRows, H - 1);
    live[u] = h0 + u * L::kRows < H;
    xh[u] = h * p.xs[side].h;
    dh[u] = h * p.ds[side].h;
    oh[u] = h * p.os[side].h;
  }
  const T* w = static_cast<const T*>(p.w[side]);
  float2 wa[kP], wb[kP], da[kP], db[kP];
  ln.weights(w, wa, wb);
#pragma unroll
  for (int e = 0; e < kP; ++e) da[e] = db[e] = make_float2(0.f, 0.f);

  struct Rows {
    uint4 x[kUnrollBwd], z[kUnrollBwd];
    Angles<T, D, kInter, kFull, kMulti> ang;
    long long out;
  };
  Pos<kMulti> pos;
  // start the loads of the walk's token and of the next one's position
  auto fetch = [&](Rows& r) {
    const T* x = x0 + st[side][0].at(wk.b, wk.n);
    const T* dz = dz0 + st[side][1].at(wk.b, wk.n);
    r.out = st[side][2].at(wk.b, wk.n);
#pragma unroll
    for (int u = 0; u < kUnrollBwd; ++u) {
      r.z[u] = ln.load(dz + dh[u]);
      if (w != nullptr) r.x[u] = ln.load(x + xh[u]);
    }
    r.ang.load(p, ln, pos);
    wk.next(p);
    if (wk.live()) pos.load(p, wk.b, wk.n);
  };
  auto work = [&](const Rows& r) {
    T* dx = dx0 + r.out;
    // dy: the transposed rotation turns the sine's sign
    float2 ya[kUnrollBwd][kP], yb[kUnrollBwd][kP];
    {
      float2 ca[kP], sa[kP], cb[kP], sb[kP];
#pragma unroll
      for (int e = 0; e < kP; ++e) {
        ca[e] = r.ang.cosine(false, e);
        cb[e] = r.ang.cosine(true, e);
        const float2 s0 = r.ang.sine(false, e), s1 = r.ang.sine(true, e);
        sa[e] = make_float2(-s0.x, -s0.y);
        sb[e] = make_float2(-s1.x, -s1.y);
      }
#pragma unroll
      for (int u = 0; u < kUnrollBwd; ++u) {
        Half<T>::unpack(r.z[u].x, r.z[u].y, ya[u]);
        Half<T>::unpack(r.z[u].z, r.z[u].w, yb[u]);
        turn<L, kInter, kFull>(ln, ya[u], yb[u], ca, sa, cb, sb);
      }
    }
    if (w != nullptr) {
      float2 fa[kUnrollBwd][kP], fb[kUnrollBwd][kP];
      float2 ga[kUnrollBwd][kP], gb[kUnrollBwd][kP];  // dy w
      float sums[2 * kUnrollBwd];                     // of x^2 and of dy w x, per row
#pragma unroll
      for (int u = 0; u < kUnrollBwd; ++u) {
        Half<T>::unpack(r.x[u].x, r.x[u].y, fa[u]);
        Half<T>::unpack(r.x[u].z, r.x[u].w, fb[u]);
        float2 ss = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < kP; ++e) {
          ga[u][e] = mul2(ya[u][e], wa[e]);
          gb[u][e] = mul2(yb[u][e], wb[e]);
          ss = fma2(fa[u][e], fa[u][e], ss);
          ss = fma2(fb[u][e], fb[u][e], ss);
          dot = fma2(ga[u][e], fa[u][e], dot);
          dot = fma2(gb[u][e], fb[u][e], dot);
        }
        sums[u] = ss.x + ss.y;
        sums[kUnrollBwd + u] = dot.x + dot.y;
      }
      static_assert(kUnrollBwd == 2, "four sums a step");
      const float mine = sum4<L::kLanes>(sums[0], sums[1], sums[2], sums[3]);
      const float r4 = rsqrtf(mine * (1.f / D) + p.eps);  // in the lanes that hold a sum of x^2
#pragma unroll
      for (int u = 0; u < kUnrollBwd; ++u) {
        const float rn = from4<L::kLanes>(r4, u), dot = from4<L::kLanes>(mine, 2 + u);
        const float k = -rn * rn * dot * (1.f / D);
        const float2 rr = make_float2(rn, rn), kk = make_float2(k, k);
        const float2 rl = live[u] ? rr : make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < kP; ++e) {
          da[e] = fma2(mul2(ya[u][e], rl), fa[u][e], da[e]);
          db[e] = fma2(mul2(yb[u][e], rl), fb[u][e], db[e]);
          ya[u][e] = mul2(rr, fma2(fa[u][e], kk, ga[u][e]));
          yb[u][e] = mul2(rr, fma2(fb[u][e], kk, gb[u][e]));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnrollBwd; ++u)
      if (live[u]) ln.store(dx + oh[u], Half<T>::pack(ya[u]), Half<T>::pack(yb[u]));
  };
  if (wk.live()) {
    Rows even, odd;
    pos.load(p, wk.b, wk.n);
    fetch(even);
    while (true) {
      if (!wk.live()) {
        work(even);
        break;
      }
      fetch(odd);
      work(even);
      if (!wk.live()) {
        work(odd);
        break;
      }
      fetch(even);
      work(odd);
    }
  }
  if (p.dw == nullptr) return;
#pragma unroll
  for (int e = 0; e < kP; ++e) {
    float* r = &red[warp * L::kRows + ln.row][ln.col + 2 * e];
    r[0] = da[e].x, r[1] = da[e].y;
    r[ln.gap] = db[e].x, r[ln.gap + 1] = db[e].y;
  }
  if ((threadIdx.x & 31) == 0) red_side[warp] = side;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps * L::kRows; ++k)
      if (red_side[k / L::kRows] == i / D) sum += red[k][i % D];
    p.dw[static_cast<size_t>(blockIdx.x) * 2 * D + i] = sum;
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
