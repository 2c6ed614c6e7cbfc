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
//   - a warp takes the same heads of many tokens: weights stay in registers, the token's table
//     columns are loaded once for all of its row loads;
//   - the row sums of an item are reduced together (each step of the exchange halves the values a
//     lane still carries), so r is computed once per row instead of once per lane and row;
//   - arithmetic is in pairs of fp32 values.
// Measured on a B200 (copy rate 6.54 TB/s), bf16, heads of 128: 16384 tokens of 32 + 8 heads 54.8 us, 6.1
// TB/s; the gradient of 8192 tokens of 16 + 16 heads 41.3 us, 4.9 TB/s (36.8 us without the weights' sum);
// 16384 tokens into a paged cache 66.5 us, 6.1 TB/s, and 64 tokens 3.2 us.  (Rates of heads that fill the tiles, 8 or
// 4 in bf16: the blocks are shared out evenly between groups of heads, whatever a group holds.)
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "common.cuh"
#include "dev/ptx_store.cuh"

namespace attn {
namespace qkn {

constexpr int kThreads = 256;  // of the paged form
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;     // row loads of a warp's item, forward
constexpr int kUnrollBwd = 2;  // backward: of x and of dz
// per SM, paged form: 80 registers a thread, which partial rotation of halves (20 bytes spilled, 40 with several axes)
// and side-by-side pairs with several axes (4) do not quite fit
constexpr int kBlocks = 3;
constexpr int kMaxAxes = 4;

// Element strides of a packed [N][H][d] view (d contiguous).
struct View {
  long long h, n;
};

struct Params {
  const void* w[2];   // weights of queries and keys [d], or null: not normalised
  const float* rope;  // [max_pos][rot]: cosines, then sines
  const int* pos;     // [axes][B][N] by the strides below
  long long pos_axis, pos_b;
  int end[kMaxAxes];  // first pair past each axis's section
  int axes, rot, max_pos;
  int B, N, H[2];
  float eps;
  float* dw;  // backward: partial weight gradients [blocks][d], or null
  // paged form: queries and keys, where the queries go, the values; tokens with a negative slot are left out
  const void* x[2];
  void* out[1];
  const void* v;
  View xs[2], os[1], vs;
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
  // this lane's halves of a row load that lies in shared memory as it does in memory
  __device__ __forceinline__ uint4 read(const uint8_t* rows) const {
    const uint8_t* p = rows + row * (D * sizeof(T)) + col * sizeof(T);
    if constexpr (kInter) {
      return *reinterpret_cast<const uint4*>(p);
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      const uint2 y = *reinterpret_cast<const uint2*>(p + gap * sizeof(T));
      return make_uint4(x.x, x.y, y.x, y.y);
    }
  }
  __device__ __forceinline__ void write(uint8_t* rows, uint2 a, uint2 b) const {
    store(reinterpret_cast<T*>(rows + row * (D * sizeof(T)) + col * sizeof(T)), a, b);
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

// r = 1 / sqrt(mean(x^2) + eps) of the kUnroll rows in raw, in the lanes where sum4 leaves a row's sum.
template <typename T, typename L>
__device__ __forceinline__ float inverse_norms(const uint4 (&raw)[kUnroll], float eps) {
  constexpr int kP = L::kP;
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
  static_assert(kUnroll == 4, "four sums a step");
  return rsqrtf(sum4<L::kLanes>(ss[0], ss[1], ss[2], ss[3]) * (1.f / (L::kLanes * 2 * L::kH)) + eps);
}

// Angle times weight, of the lane's columns and for their partners.
template <typename L, bool kInter>
struct Coeffs {
  static constexpr int kP = L::kP;
  float2 ca[kP], sa[kP], cb[kP], sb[kP];
  template <typename A>
  __device__ __forceinline__ Coeffs(const A& ang, const float2 (&wa)[kP], const float2 (&wb)[kP]) {
#pragma unroll
    for (int e = 0; e < kP; ++e) {
      ca[e] = mul2(wa[e], ang.cosine(false, e));
      cb[e] = mul2(wb[e], ang.cosine(true, e));
      sa[e] = mul2(kInter ? swap2(wa[e]) : wb[e], ang.sine(false, e));
      sb[e] = mul2(kInter ? swap2(wb[e]) : wa[e], ang.sine(true, e));
    }
  }
};

// ------------------------------------------------------------------------------------------
// Paged form: rows by ordinary loads, because tokens are left out and go to scattered rows
// ------------------------------------------------------------------------------------------
// Strides that every token needs again: kept in shared memory and read there each time, so that they
// do not hold registers through the loop (which runs at 80 registers, three blocks per SM).
struct Strides {
  long long n;
  __device__ __forceinline__ void set(const View& v) volatile { n = v.n; }
  __device__ __forceinline__ long long at(int in) const volatile { return in * n; }
};

// bf16, packed tokens (B = 1).  A warp takes the same heads (queries, keys or values) of every step-th
// token; the next token's position and slot are on their way while it works on the current one.
template <typename T, int D, bool kInter, bool kFull, bool kMulti>
__global__ void __launch_bounds__(kThreads, kBlocks) qk_norm_rope_paged_kernel(const Params p) {
  using L = Lane<T, D, kInter, kFull>;
  constexpr int kP = L::kP;
  __shared__ volatile Strides st[4];  // of a kind's input, of the queries' output
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) st[i].set(p.xs[i]);
    st[2].set(p.vs);
    st[3].set(p.os[0]);
  }
  __syncthreads();
  const L ln(p.rot);
  constexpr int kHeads = kUnroll * L::kRows;
  const int cq = (p.H[0] + kHeads - 1) / kHeads, ck = (p.H[1] + kHeads - 1) / kHeads, chunks = cq + 2 * ck;
  const int warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int step = gridDim.x * kWarps / chunks;  // the launch has chunks warps at least
  const int chunk = warp % chunks;
  int n = warp / chunks;
  if (n >= step || n >= p.N) return;
  const int kind = chunk < cq ? 0 : chunk < cq + ck ? 1 : 2, side = kind == 0 ? 0 : 1;
  const bool copy = kind == 2;  // values: as they are
  const int h0 = (chunk - (kind == 0 ? 0 : kind == 1 ? cq : cq + ck)) * kHeads + ln.row, H = p.H[side];
  const View& xs = copy ? p.vs : p.xs[side];
  const T* x0 = static_cast<const T*>(copy ? p.v : p.x[side]) + h0 * xs.h + ln.col;
  T* out0 = kind != 0 ? static_cast<T*>(p.cache[kind - 1]) + h0 * D + ln.col
                      : static_cast<T*>(p.out[0]) + h0 * p.os[0].h + ln.col;
  const long long xh = xs.h * L::kRows, oh = (kind != 0 ? D : p.os[0].h) * L::kRows;
  const T* w = copy ? nullptr : static_cast<const T*>(p.w[side]);
  float2 wa[kP], wb[kP];
  ln.weights(w, wa, wb);
  // the cache slot of a token (below 0: left out)
  auto slot_of = [&](int t) -> int {
    const int s = __ldg(p.slots + t);
    if (s < p.slots_total) return s;
    atomicExch(&g_device_error, ATTN_ERR_INVALID_ARG);
    return -1;
  };
  Pos<kMulti> pos;
  if (!copy) pos.load(p, 0, n);
  int slot = slot_of(n);
  while (true) {
    const int cur = slot, cn = n;
    const Pos<kMulti> cur_pos = pos;
    const bool more = p.N - n > step;
    n += step;
    uint4 raw[kUnroll];
    if (cur >= 0) {
      const T* x = x0 + st[kind].at(cn);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        raw[u] = h0 + u * L::kRows < H ? ln.load(x + u * xh) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (more) {
      if (!copy) pos.load(p, 0, n);
      slot = slot_of(n);
    }
    if (cur >= 0) {
      T* out = kind != 0 ? out0 + static_cast<long long>(cur) * p.H[1] * D : out0 + st[3].at(cn);
      if (copy) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (h0 + u * L::kRows < H)
            ln.store(out + u * oh, make_uint2(raw[u].x, raw[u].y), make_uint2(raw[u].z, raw[u].w));
      } else {
        Angles<T, D, kInter, kFull, kMulti> ang;
        ang.load(p, ln, cur_pos);
        const Coeffs<L, kInter> k(ang, wa, wb);
        const float r4 = w != nullptr ? inverse_norms<T, L>(raw, p.eps) : 1.f;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const float r = from4<L::kLanes>(r4, u);
          const float2 rr = make_float2(r, r);
          float2 fa[kP], fb[kP];
          Half<T>::unpack(raw[u].x, raw[u].y, fa);
          Half<T>::unpack(raw[u].z, raw[u].w, fb);
          turn<L, kInter, kFull>(ln, fa, fb, k.ca, k.sa, k.cb, k.sb);
#pragma unroll
          for (int e = 0; e < kP; ++e) fa[e] = mul2(fa[e], rr), fb[e] = mul2(fb[e], rr);
          if (h0 + u * L::kRows < H) ln.store(out + u * oh, Half<T>::pack(fa), Half<T>::pack(fb));
        }
      }
    }
    if (!more) break;
  }
}

// ------------------------------------------------------------------------------------------
// Dense and packed form, and the gradient: tiles of kTokens tokens x a few heads by TMA
// ------------------------------------------------------------------------------------------
// A block of four warps streams tiles through a ring in shared memory: one thread starts the load of
// the tile after next, each warp works on one token of the current tile in place, and the result
// leaves from the same buffer by one TMA store.  The tensor maps carry all strides (those of a fused
// projection, of head-major or token-major outputs, 0 for broadcast heads), and clip heads and
// tokens past the last.  So a thread holds no addresses and fits 72 registers: 28 warps per SM with
// two tiles a block on their way.  (Rows by ordinary loads with the next ones in registers: 65 us
// instead of 54.8, the moves wait for the loads; a fourth stage, which costs a block per SM: 57.3.)
// A block's tiles all have the same heads.
constexpr int kTokens = 4;
constexpr int kTileThreads = 32 * kTokens;
constexpr int kTileBlocks = 7;     // per SM: 72 registers a thread (bf16: 4 to 12 bytes spilled in three of the eight forms)
constexpr int kTileBlocksBwd = 5;  // backward: 96 (8 bytes spilled by partial rotation of halves with several axes, none
                                   // else; 6 blocks at 80 spill more: 2% slower with several axes, else the same)
constexpr int kStages = 3;
constexpr int kWarpBytes = 2048;  // of a stage: a warp's rows (backward: half of them x, half dz)
constexpr int kStageBytes = kTokens * kWarpBytes;

struct __align__(128) TileSmem {
  uint8_t stage[kStages][kStageBytes];
  uint64_t full[kStages];
  int abort;
};

__device__ __forceinline__ void tile_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int h, int n, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(h), "r"(n), "r"(b)
      : "memory");
}
__device__ __forceinline__ void tile_store(const CUtensorMap* map, uint32_t src, int h, int n, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(0), "r"(h), "r"(n), "r"(b)
      : "memory");
}

// The tiles of a block: the same heads, every step-th run of kTokens tokens.
struct Tiles {
  int side, h0;   // queries or keys, first head
  int left;       // runs from the current one to the end
  int step, step_b, step_r, runs;
  int b, r;       // batch row and run of the current tile
  __device__ __forceinline__ Tiles(const Params& p, int heads) {
    const int cq = (p.H[0] + heads - 1) / heads, chunks = cq + (p.H[1] + heads - 1) / heads;
    const int chunk = blockIdx.x % chunks, first = blockIdx.x / chunks;
    side = chunk < cq ? 0 : 1;
    h0 = (chunk - (side ? cq : 0)) * heads;
    step = gridDim.x / chunks;  // a whole number: the launch sees to it
    runs = (p.N + kTokens - 1) / kTokens;
    left = p.B * runs - first;
    b = first / runs;
    r = first % runs;
    step_b = step / runs;
    step_r = step % runs;
  }
  __device__ __forceinline__ bool live() const { return left > 0; }
  __device__ __forceinline__ int n() const { return r * kTokens; }
  __device__ __forceinline__ void next() {
    left -= step;
    b += step_b;
    r += step_r;
    if (r >= runs) {
      r -= runs;
      ++b;
    }
  }
};

// What both kernels do around a tile's arithmetic.  kInputs tensors of kBytes each per stage; the result
// replaces the last of them.
template <typename Work>
__device__ __forceinline__ void stream_tiles(TileSmem& sm, Tiles tl, const CUtensorMap* in0, const CUtensorMap* in1,
                                             const CUtensorMap* out, uint32_t bytes, Work&& work) {
  const uint32_t base = dev::smem_u32(sm.stage[0]);
  volatile int* abort = &sm.abort;
  // start the load of tile number j of the block
  auto load = [&](int j, const Tiles& t) {
    if (!t.live()) return;
    const int s = j % kStages;
    const uint32_t bar = dev::smem_u32(&sm.full[s]), dst = base + s * kStageBytes;
    dev::mbar_arrive_expect_tx(bar, in1 != nullptr ? 2 * bytes : bytes);
    tile_load(dst, in0, bar, t.h0, t.n(), t.b);
    if (in1 != nullptr) tile_load(dst + bytes, in1, bar, t.h0, t.n(), t.b);
  };
  if (threadIdx.x == 0) {
    Tiles t = tl;
    for (int j = 0; j < kStages - 1; ++j, t.next()) load(j, t);
  }
  const uint32_t from = in1 != nullptr ? bytes : 0;
  bool ok = true;
  int i = 0;
  for (; tl.live(); ++i, tl.next()) {
    const int s = i % kStages;
    // (a warp gives up as a whole: the work behind the wait exchanges values between its lanes)
    ok = work(sm.stage[s], tl, [&] {
      return __all_sync(0xffffffffu, wait_bounded(dev::smem_u32(&sm.full[s]), (i / kStages) & 1, abort)) != 0;
    });
    dev::fence_proxy_async_smem();
    ok = __syncthreads_and(ok) != 0;
    if (!ok) break;
    if (threadIdx.x == 0) {
      tile_store(out, base + s * kStageBytes + from, tl.h0, tl.n(), tl.b);
      dev::bulk_commit_group();
      dev::bulk_wait_group_read1();  // the tile before has left its stage: the one after next may come
      Tiles t = tl;
      for (int j = 0; j < kStages - 1; ++j) t.next();
      load(i + kStages - 1, t);
    }
  }
  if (threadIdx.x == 0) {
    dev::bulk_wait_group_read0();
    if (!ok) {  // a wait gave up: the tiles from i on may still be landing
      for (int j = i; j < i + kStages - 1 && tl.live(); ++j, tl.next())
        wait_drain(dev::smem_u32(&sm.full[j % kStages]), (j / kStages) & 1);
    }
  }
}

__device__ __forceinline__ void init_tiles(TileSmem& sm) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) dev::mbar_init(dev::smem_u32(&sm.full[s]), 1);
    sm.abort = 0;
    dev::fence_barrier_init();
  }
  __syncthreads();
}

// Forward.
template <typename T, int D, bool kInter, bool kFull, bool kMulti>
__global__ void __launch_bounds__(kTileThreads, kTileBlocks)
    qk_norm_rope_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_qo, const __grid_constant__ CUtensorMap tm_ko,
                        const Params p) {
  using L = Lane<T, D, kInter, kFull>;
  constexpr int kP = L::kP;
  __shared__ TileSmem sm;
  init_tiles(sm);
  const L ln(p.rot);
  const Tiles tl(p, kUnroll * L::kRows);
  const int warp = threadIdx.x >> 5;
  const T* w = static_cast<const T*>(p.w[tl.side]);
  float2 wa[kP], wb[kP];
  ln.weights(w, wa, wb);
  stream_tiles(sm, tl, tl.side ? &tm_k : &tm_q, nullptr, tl.side ? &tm_ko : &tm_qo, kStageBytes,
               [&](uint8_t* stage, const Tiles& t, auto&& wait) {
                 const int n = t.n() + warp;
                 uint8_t* rows = stage + warp * kWarpBytes;
                 Angles<T, D, kInter, kFull, kMulti> ang;
                 if (n < p.N) {
                   Pos<kMulti> pos;
                   pos.load(p, t.b, n);
                   ang.load(p, ln, pos);
                 }
                 if (!wait()) return false;
                 if (n < p.N) {
                   const Coeffs<L, kInter> k(ang, wa, wb);
                   uint4 raw[kUnroll];
#pragma unroll
                   for (int u = 0; u < kUnroll; ++u) raw[u] = ln.read(rows + u * 512);
                   const float r4 = w != nullptr ? inverse_norms<T, L>(raw, p.eps) : 1.f;
#pragma unroll
                   for (int u = 0; u < kUnroll; ++u) {
                     const float r = from4<L::kLanes>(r4, u);
                     const float2 rr = make_float2(r, r);
                     float2 fa[kP], fb[kP];
                     Half<T>::unpack(raw[u].x, raw[u].y, fa);
                     Half<T>::unpack(raw[u].z, raw[u].w, fb);
                     turn<L, kInter, kFull>(ln, fa, fb, k.ca, k.sa, k.cb, k.sb);
#pragma unroll
                     for (int e = 0; e < kP; ++e) fa[e] = mul2(fa[e], rr), fb[e] = mul2(fb[e], rr);
                     ln.write(rows + u * 512, Half<T>::pack(fa), Half<T>::pack(fb));
                   }
                 }
                 return true;
               });
}

// Backward: the tile's x and dz, dx in place of dz; a warp keeps the weight gradient of its columns in
// registers, and a block adds its warps' up in a fixed order into one partial row.
template <typename T, int D, bool kInter, bool kFull, bool kMulti>
__global__ void __launch_bounds__(kTileThreads, kTileBlocksBwd)
    qk_norm_rope_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_gq, const __grid_constant__ CUtensorMap tm_gk,
                            const __grid_constant__ CUtensorMap tm_dq, const __grid_constant__ CUtensorMap tm_dk,
                            const Params p) {
  using L = Lane<T, D, kInter, kFull>;
  constexpr int kP = L::kP;
  __shared__ TileSmem sm;
  init_tiles(sm);
  const L ln(p.rot);
  const Tiles tl(p, kUnrollBwd * L::kRows);
  const int warp = threadIdx.x >> 5;
  const T* w = static_cast<const T*>(p.w[tl.side]);
  const bool weighted = w != nullptr;
  float2 wa[kP], wb[kP], da[kP], db[kP];
  ln.weights(w, wa, wb);
#pragma unroll
  for (int e = 0; e < kP; ++e) da[e] = db[e] = make_float2(0.f, 0.f);
  const CUtensorMap* mx = tl.side ? &tm_k : &tm_q;
  const CUtensorMap* mz = tl.side ? &tm_gk : &tm_gq;
  stream_tiles(sm, tl, weighted ? mx : mz, weighted ? mz : nullptr, tl.side ? &tm_dk : &tm_dq, kStageBytes / 2,
               [&](uint8_t* stage, const Tiles& t, auto&& wait) {
                 const int n = t.n() + warp;
                 const uint8_t* xrows = stage + warp * (kWarpBytes / 2);
                 uint8_t* zrows = stage + (weighted ? kStageBytes / 2 : 0) + warp * (kWarpBytes / 2);
                 Angles<T, D, kInter, kFull, kMulti> ang;
                 if (n < p.N) {
                   Pos<kMulti> pos;
                   pos.load(p, t.b, n);
                   ang.load(p, ln, pos);
                 }
                 if (!wait()) return false;
                 if (n >= p.N) return true;
                 // dy: the transposed rotation turns the sine's sign
                 float2 ya[kUnrollBwd][kP], yb[kUnrollBwd][kP];
                 {
                   float2 ca[kP], sa[kP], cb[kP], sb[kP];
#pragma unroll
                   for (int e = 0; e < kP; ++e) {
                     ca[e] = ang.cosine(false, e);
                     cb[e] = ang.cosine(true, e);
                     const float2 s0 = ang.sine(false, e), s1 = ang.sine(true, e);
                     sa[e] = make_float2(-s0.x, -s0.y);
                     sb[e] = make_float2(-s1.x, -s1.y);
                   }
#pragma unroll
                   for (int u = 0; u < kUnrollBwd; ++u) {
                     const uint4 raw = ln.read(zrows + u * 512);
                     Half<T>::unpack(raw.x, raw.y, ya[u]);
                     Half<T>::unpack(raw.z, raw.w, yb[u]);
                     turn<L, kInter, kFull>(ln, ya[u], yb[u], ca, sa, cb, sb);
                   }
                 }
                 if (weighted) {
                   uint4 raw[kUnrollBwd];
                   float sums[2 * kUnrollBwd];  // of x^2 and of dy w x, per row
#pragma unroll
                   for (int u = 0; u < kUnrollBwd; ++u) {
                     raw[u] = ln.read(xrows + u * 512);
                     float2 fa[kP], fb[kP];
                     Half<T>::unpack(raw[u].x, raw[u].y, fa);
                     Half<T>::unpack(raw[u].z, raw[u].w, fb);
                     float2 ss = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
#pragma unroll
                     for (int e = 0; e < kP; ++e) {
                       ss = fma2(fa[e], fa[e], ss);
                       ss = fma2(fb[e], fb[e], ss);
                       dot = fma2(mul2(ya[u][e], wa[e]), fa[e], dot);
                       dot = fma2(mul2(yb[u][e], wb[e]), fb[e], dot);
                     }
                     sums[u] = ss.x + ss.y;
                     sums[kUnrollBwd + u] = dot.x + dot.y;
                   }
                   static_assert(kUnrollBwd == 2, "four sums a step");
                   const float mine = sum4<L::kLanes>(sums[0], sums[1], sums[2], sums[3]);
                   const float r4 = rsqrtf(mine * (1.f / D) + p.eps);  // in the lanes that hold a sum of x^2
                   const int heads = p.H[tl.side] - tl.h0 - ln.row;
#pragma unroll
                   for (int u = 0; u < kUnrollBwd; ++u) {
                     const float r = from4<L::kLanes>(r4, u), dot = from4<L::kLanes>(mine, 2 + u);
                     const float k = -r * r * dot * (1.f / D);
                     const float2 rr = make_float2(r, r), kk = make_float2(k, k);
                     float2 fa[kP], fb[kP];
                     Half<T>::unpack(raw[u].x, raw[u].y, fa);
                     Half<T>::unpack(raw[u].z, raw[u].w, fb);
                     // rows past the last head are zeros and add nothing (0 x infinity for eps = 0: hence rl)
                     const float2 rl = u * L::kRows < heads ? rr : make_float2(0.f, 0.f);
#pragma unroll
                     for (int e = 0; e < kP; ++e) {
                       da[e] = fma2(mul2(ya[u][e], rl), fa[e], da[e]);
                       db[e] = fma2(mul2(yb[u][e], rl), fb[e], db[e]);
                       ya[u][e] = mul2(rr, fma2(fa[e], kk, mul2(ya[u][e], wa[e])));
                       yb[u][e] = mul2(rr, fma2(fb[e], kk, mul2(yb[u][e], wb[e])));
                     }
                   }
                 }
#pragma unroll
                 for (int u = 0; u < kUnrollBwd; ++u)
                   ln.write(zrows + u * 512, Half<T>::pack(ya[u]), Half<T>::pack(yb[u]));
                 return true;
               });
  if (p.dw != nullptr) {
    // the ring becomes the block's buffer of column sums [kTokens * kRows][D]
    static_assert(kTokens * L::kRows * D * sizeof(float) <= sizeof(sm.stage), "column sums");
    __syncthreads();
    float(*red)[D] = reinterpret_cast<float(*)[D]>(&sm.stage[0][0]);
#pragma unroll
    for (int e = 0; e < kP; ++e) {
      float* r = &red[warp * L::kRows + ln.row][ln.col + 2 * e];
      r[0] = da[e].x, r[1] = da[e].y;
      r[ln.gap] = db[e].x, r[ln.gap + 1] = db[e].y;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kTileThreads) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < kTokens * L::kRows; ++k) sum += red[k][i];
      p.dw[static_cast<size_t>(blockIdx.x) * D + i] = sum;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Sum of the blocks' partial weight gradients, in a fixed order.  Block g of chunks holds queries for
// g % chunks < cq, else keys.  A block of 8 columns x 128 rows at a time; grid (d / 8, 2).
constexpr int kSumRows = 128;
__global__ void __launch_bounds__(8 * kSumRows)
    qk_norm_dw_kernel(const float* __restrict__ part, int blocks, int chunks, int cq, int d, float* dwq, float* dwk) {
  __shared__ float red[32][9];
  float* out = blockIdx.y == 0 ? dwq : dwk;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = threadIdx.x & 7, k = threadIdx.x >> 3;
  // this side's rows in order, n of every `chunks`; this thread takes every kSumRows-th, from the k-th on
  const int n = max(blockIdx.y == 0 ? cq : chunks - cq, 1);
  const int step_g = kSumRows / n, step_c = kSumRows % n;
  int g = k / n, c = k % n;
  const int end = blocks / chunks;
  const float* at = part + (blockIdx.y == 0 ? 0 : cq) * d + blockIdx.x * 8 + i;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float t = 0.f;
  while (g < end) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      v[u] = g < end ? __ldcg(at + static_cast<size_t>(g * chunks + c) * d) : 0.f;
      g += step_g, c += step_c;
      if (c >= n) c -= n, ++g;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) t += v[u];
  }
  // the four rows of a warp, then the warps: warp w sums column w
  t += __shfl_xor_sync(0xffffffffu, t, 8);
  t += __shfl_xor_sync(0xffffffffu, t, 16);
  if (lane < 8) red[warp][lane] = t;
  __syncthreads();
  if (warp >= 8) return;
  t = red[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (lane == 0) out[blockIdx.x * 8 + warp] = t;
}

}  // namespace qkn
}  // namespace attn
