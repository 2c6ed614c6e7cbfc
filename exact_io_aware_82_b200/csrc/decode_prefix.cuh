// Decode for a batch whose sequences share long prefixes, over a paged KV cache: the keys of a
// prefix are read once for all the sequences behind it, those of a sequence's own pages once for
// that sequence, and the two parts are joined exactly by their log-sum-exps.
//
// The mathematics is that of decode.cuh: with the keys of one query row split into parts, part s
// gives O_s = sum_j 2^(x_j - m_s) v_j / l_s and lse_s = ln(sum exp); then LSE = ln sum_s
// exp(lse_s) and O = sum_s exp(lse_s - LSE) O_s.
//
// Work.  A job is one kv head of either a block of sequences of one group (their query rows
// against the prefix keys) or one sequence (its G query rows against its own keys); a step is one
// 128-key tile of a job.  Query rows are the M = 128 rows of a tensor-core product, S = Q K^T and
// O += P V with P taken from tensor memory:
//   both mode   a block of more than 128 query rows: two row tiles take every step, so a key
//               tile read once feeds up to 256 rows;
//   alt mode    up to 128 rows: the two row tiles hold the same rows and take alternate steps, so
//               one step's softmax overlaps the next step's products; the two halves of the
//               keys end as two parts.
// All steps of all jobs stand in one line, weighted by what a step costs, and every CTA takes an
// equal length of it (persistent, one CTA per SM): long prefixes are cut over many CTAs, short
// sequences are taken several to a CTA, and compute-bound prefix steps run beside the
// memory-bound steps of the sequences.  The cuts follow from the lengths alone, which each CTA
// sums up for itself when it starts, so there is no counter and no order of arrival: results are
// the same in every run, and launches share nothing but the caller's workspace.
//
// Warps (12): 0-3 softmax and epilogue of row tile 0, 4-7 of row tile 1 (thread = row = TMEM
// lane), 8 the tcgen05.mma issuer (all lanes zero the value rows past a job's last key first:
// what a page holds there may be infinite or NaN, and 0 x NaN would reach the sum), 9 the job walk
// and the TMA producer (one lane per box: a 128-key tile is 128 / min(page size, 128) pieces x 2
// column halves), 10-11 idle.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "dev/ptx_store.cuh"

namespace attn {
namespace pfx {

constexpr int kD = 128;
constexpr int kTile = 128;
constexpr int kThreads = 384;
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp = 9;
constexpr uint32_t kRegsLaunch = 168;
constexpr uint32_t kRegsSoftmax = 208;
constexpr uint32_t kRegsOther = 88;
static_assert(2 * kRegsSoftmax + kRegsOther == 3 * kRegsLaunch, "register split must balance");
constexpr uint32_t kTileBytes = kTile * kD * 2;
constexpr uint32_t kHalfBytes = kTile * 64 * 2;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

// Cost of a step and of a job (in arbitrary equal units) on the line the CTAs share out.
constexpr int kCostBoth = 4;
constexpr int kCostAlt = 3;
constexpr int kCostJob = 2;

// Rows of partial results: a block of n sequences starts its jobs' rows at 2 G Hkv (its first
// sequence) + 2 G n (its kv head), a sequence's own job at 2 G (its job number), and every CTA
// adds its index times kCtaRows (2 G): consecutive segments on the line never overlap.
constexpr int kCtaRows = 256;

struct Params {
  int B, Hq, Hkv, G, S;  // S = 128 / G: sequences in one row tile
  int num_groups, max_prefix_len, max_prefix_pages;
  int max_seq_len, max_pages;
  int num_pages, page_shift;
  const int* prefix_table;  // [num_groups][max_prefix_pages]
  const int* prefix_lens;   // [num_groups]
  const int* group_starts;  // [num_groups + 1]
  const int* block_table;   // [B][max_pages]
  const int* seq_lens;      // [B]
  float c;                  // scale * log2(e), never 0
  float* ws_o;              // partial outputs [rows][128], then
  float* ws_lse;            // their log-sum-exps [rows]
  int* plan;                // [0] cost per CTA, [1] cost of all prefix jobs, then the cost before
                            // each group [num_groups] and before each sequence [B]
  long long own_row0;       // first row of the sequences' own parts
};

// ---- the line of jobs (shared with the combine kernel) ----
struct Group {
  int b0, n, tiles;  // first sequence, sequences, key tiles
  int full;          // blocks of 2 S sequences
  int rest;          // sequences of the last, smaller block
  int len;
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return max(lo, min(x, hi)); }

__device__ __forceinline__ Group load_group(const Params& p, int g) {
  Group r;
  r.b0 = clampi(__ldg(p.group_starts + g), 0, p.B);
  r.n = clampi(__ldg(p.group_starts + g + 1), r.b0, p.B) - r.b0;
  r.len = clampi(__ldg(p.prefix_lens + g), 0, p.max_prefix_len);
  r.tiles = (r.len + kTile - 1) / kTile;
  r.full = r.n / (2 * p.S);
  r.rest = r.n % (2 * p.S);
  return r;
}

__device__ __forceinline__ int job_cost(int tiles, int weight) {
  return tiles > 0 ? tiles * weight + kCostJob : 0;
}
__device__ __forceinline__ int rest_weight(const Params& p, const Group& g) {
  return g.rest > p.S ? kCostBoth : kCostAlt;
}
// one kv head of all blocks of a group, times the kv heads
__device__ __forceinline__ int group_cost(const Params& p, const Group& g) {
  const int rest = g.rest > 0 ? job_cost(g.tiles, rest_weight(p, g)) : 0;
  return p.Hkv * (g.full * job_cost(g.tiles, kCostBoth) + rest);
}
__device__ __forceinline__ int seq_len(const Params& p, int b) {
  return clampi(__ldg(p.seq_lens + b), 0, p.max_seq_len);
}
__device__ __forceinline__ int seq_cost(const Params& p, int b) {
  return p.Hkv * job_cost((seq_len(p, b) + kTile - 1) / kTile, kCostAlt);
}
// first step at or after position x of the line, for a job at position c with steps of weight w
__device__ __forceinline__ int step_at(int x, int c, int w) { return x <= c ? 0 : (x - c + w - 1) / w; }

// One segment: a CTA's run of steps of one job.
struct Unit {
  int valid;
  int both;        // 1: both row tiles take every step; 0: alternate steps
  int flip;        // alt mode: the row tile that takes the first step
  int nk;          // steps
  int tail;        // keys of the last step (1..128)
  int rows[2];     // real query rows of each row tile
  long long out[2];  // first partial row of each row tile
  int b0, hk;      // first sequence, kv head
  int own;         // 1: a sequence's own keys
  int key0, len;   // first key, keys of the job
  const int* table;
  int table_pages;
};

struct __align__(1024) Smem {
  uint8_t q[2][kTileBytes];
  uint8_t k[2][kTileBytes];
  uint8_t v[2][kTileBytes];
  uint8_t stage[8][4096];  // per softmax warp: 32 rows x 32 fp32 columns on their way out
  uint64_t bar_q, bar_qempty;
  uint64_t bar_kfull[2], bar_kempty[2], bar_vfull[2], bar_vempty[2];
  uint64_t bar_s[2], bar_p[2], bar_o[2], bar_drain;
  uint64_t bar_unit_full[2], bar_unit_empty[2];
  Unit unit[2];
  int scan[2][kThreads / 32 + 1];
  int start[4];  // where this CTA's share begins: kind, group / sequence, position of its cost, -
  uint32_t tmem_base;
  int abort;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");
constexpr uint32_t kUnitReaders = 9;  // 8 softmax warps, the MMA warp

// Exclusive sum over the CTA of one value per thread; every thread gets the total too.
__device__ __forceinline__ int block_scan(int v, int* buf, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the buffer's earlier readers are done
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int s = buf[w];
    if (w < warp) before += s;
    total += s;
  }
  return before + x - v;
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// kNeg: the scale is negative, so the largest scaled score comes from the smallest raw score.
template <bool kNeg>
__global__ void __launch_bounds__(kThreads, 1)
    decode_prefix_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_q_own,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;

  // ---- set-up ----
  if (tid == 0) {
    dev::mbar_init(dev::smem_u32(&sm.bar_q), 1);
    dev::mbar_init(dev::smem_u32(&sm.bar_qempty), 1);
    for (int s = 0; s < 2; ++s) {
      dev::mbar_init(dev::smem_u32(&sm.bar_kfull[s]), 1);
      dev::mbar_init(dev::smem_u32(&sm.bar_kempty[s]), 1);
      dev::mbar_init(dev::smem_u32(&sm.bar_vfull[s]), 1);
      dev::mbar_init(dev::smem_u32(&sm.bar_vempty[s]), 1);
      dev::mbar_init(dev::smem_u32(&sm.bar_s[s]), 1);
      dev::mbar_init(dev::smem_u32(&sm.bar_p[s]), 4);
      dev::mbar_init(dev::smem_u32(&sm.bar_o[s]), 1);
      dev::mbar_init(dev::smem_u32(&sm.bar_unit_full[s]), 1);
      dev::mbar_init(dev::smem_u32(&sm.bar_unit_empty[s]), kUnitReaders);
    }
    dev::mbar_init(dev::smem_u32(&sm.bar_drain), 1);
    sm.abort = 0;
    sm.start[0] = 2;  // nothing
    dev::fence_barrier_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    dev::tma_prefetch_desc(&tm_q);
    dev::tma_prefetch_desc(&tm_q_own);
    dev::tma_prefetch_desc(&tm_k);
    dev::tma_prefetch_desc(&tm_v);
  }
  if (warp == kMmaWarp) {
    dev::tmem_alloc(dev::smem_u32(&sm.tmem_base), 512);
    dev::tmem_relinquish();
  }
  // ---- this CTA's share of the line: total cost, then the job its start falls into ----
  int sum = 0, cost_prefix, cost_all;
  for (int g = tid; g < p.num_groups; g += kThreads) sum += group_cost(p, load_group(p, g));
  block_scan(sum, sm.scan[0], cost_prefix);
  sum = 0;
  for (int b = tid; b < p.B; b += kThreads) sum += seq_cost(p, b);
  block_scan(sum, sm.scan[1], cost_all);
  cost_all += cost_prefix;
  // every CTA between a job's first and last holds at least one of its steps: a share is not
  // shorter than a step
  const int share = max((cost_all + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x), kCostBoth);
  const long long lo64 = static_cast<long long>(cta) * share;
  const int lo = static_cast<int>(min(lo64, static_cast<long long>(cost_all)));
  const int hi = static_cast<int>(min(lo64 + share, static_cast<long long>(cost_all)));
  const bool plan_writer = cta == 0;
  if (plan_writer && tid == 0) {
    p.plan[0] = share;
    p.plan[1] = cost_prefix;
  }
  if (plan_writer || lo < cost_prefix) {
    int base = 0;
    for (int g0 = 0; g0 < p.num_groups; g0 += kThreads) {
      const int g = g0 + tid;
      const int cost = g < p.num_groups ? group_cost(p, load_group(p, g)) : 0;
      int total;
      const int at = base + block_scan(cost, sm.scan[0], total);
      if (plan_writer && g < p.num_groups) p.plan[2 + g] = at;
      if (cost > 0 && lo >= at && lo < at + cost) {
        sm.start[0] = 0;
        sm.start[1] = g;
        sm.start[2] = at;
      }
      base += total;
    }
  }
  if (plan_writer || lo >= cost_prefix) {
    int base = cost_prefix;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      const int b = b0 + tid;
      const int cost = b < p.B ? seq_cost(p, b) : 0;
      int total;
      const int at = base + block_scan(cost, sm.scan[1], total);
      if (plan_writer && b < p.B) p.plan[2 + p.num_groups + b] = at;
      if (cost > 0 && lo >= at && lo < at + cost) {
        sm.start[0] = 1;
        sm.start[1] = b;
        sm.start[2] = at;
      }
      base += total;
    }
  }
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;

  if (warp >= 8) {
    dev::regs_decrease<kRegsOther>();
    if (warp == kLoadWarp) {
      // ======================= job walk + TMA producer (whole warp) =======================
      int published = 0, q_loads = 0, k_issued = 0, v_issued = 0;
      bool ok = true;
      const int psize = 1 << p.page_shift;
      const int piece = psize < kTile ? psize : kTile;
      const int pieces = kTile / piece;
      const int my_piece = lane >> 1, my_half = lane & 1;
      const long long rows_total = static_cast<long long>(p.num_pages) << p.page_shift;

      // publish one segment and stream its tiles
      auto segment = [&](Unit& u) {
        const int slot = published & 1;
        if (published >= 2)
          ok = wait_bounded(dev::smem_u32(&sm.bar_unit_empty[slot]), ((published - 2) >> 1) & 1, abort);
        if (!(ok = __all_sync(0xffffffffu, ok))) return;
        u.flip = u.both ? 0 : published & 1;
        if (lane == 0) {
          sm.unit[slot] = u;
          __threadfence_block();
          dev::mbar_arrive(dev::smem_u32(&sm.bar_unit_full[slot]));
        }
        __syncwarp();
        ++published;
        // Q once the previous segment's last S products have read the Q buffers
        if (q_loads > 0) ok = wait_bounded(dev::smem_u32(&sm.bar_qempty), (q_loads - 1) & 1, abort);
        if (!(ok = __all_sync(0xffffffffu, ok))) return;
        if (lane == 0) {
          const uint32_t bq = dev::smem_u32(&sm.bar_q);
          const int tiles = u.both ? 2 : 1;
          dev::mbar_arrive_expect_tx(bq, u.own ? p.G * 256u : tiles * kTileBytes);
          for (int t = 0; t < tiles; ++t)
            for (int half = 0; half < 2; ++half)
              dev::tma_load_3d(dev::smem_u32(sm.q[t]) + half * kHalfBytes, u.own ? &tm_q_own : &tm_q,
                               bq, half * 64, u.hk * p.G, u.b0 + t * p.S);
        }
        __syncwarp();
        ++q_loads;
        // first row of this lane's piece of tile j, as a row of the page pool (-1: the piece is
        // past the last key)
        auto page_of = [&](int j) {
          const int key = u.key0 + j * kTile + my_piece * piece;
          if (j >= u.nk || my_piece >= pieces || key >= u.len) return -2;
          const int lp = key >> p.page_shift;
          return lp < u.table_pages ? __ldg(u.table + lp) : -1;
        };
        int page = page_of(0);
        for (int j = 0; ok && j < u.nk; ++j) {
          const int cur = page;
          page = page_of(j + 1);
          const int key = u.key0 + j * kTile + my_piece * piece;
          const int s = k_issued & 1;
          const uint32_t ph = ((k_issued >> 1) & 1) ^ 1;
          // pieces that hold a key of the job
          const int live = min(pieces, (u.len - u.key0 - j * kTile + piece - 1) / piece);
          const uint32_t bytes = static_cast<uint32_t>(live) * piece * 256u;
          int row = static_cast<int>(rows_total);  // a page outside the cache: reads as zero
          if (cur >= 0 && cur < p.num_pages)
            row = (cur << p.page_shift) + (key & (psize - 1));
          else if (cur != -2)
            atomicExch(&g_device_error, ATTN_ERR_INVALID_ARG);
          ok = wait_bounded(dev::smem_u32(&sm.bar_kempty[s]), ph, abort);
          if (!(ok = __all_sync(0xffffffffu, ok))) return;
          const uint32_t bk = dev::smem_u32(&sm.bar_kfull[s]);
          if (lane == 0) dev::mbar_arrive_expect_tx(bk, bytes);
          __syncwarp();
          if (cur != -2)
            dev::tma_load_3d(dev::smem_u32(sm.k[s]) + my_half * kHalfBytes + my_piece * piece * 128,
                             &tm_k, bk, my_half * 64, row, u.hk);
          ++k_issued;
          ok = wait_bounded(dev::smem_u32(&sm.bar_vempty[s]), ph, abort);
          if (!(ok = __all_sync(0xffffffffu, ok))) return;
          const uint32_t bv = dev::smem_u32(&sm.bar_vfull[s]);
          if (lane == 0) dev::mbar_arrive_expect_tx(bv, bytes);
          __syncwarp();
          if (cur != -2)
            dev::tma_load_3d(dev::smem_u32(sm.v[s]) + my_half * kHalfBytes + my_piece * piece * 128,
                             &tm_v, bv, my_half * 64, row, u.hk);
          ++v_issued;
        }
      };
      // the steps of the job at position c that belong to this CTA
      auto job = [&](Unit& u, int c, int tiles, int w) {
        const int k0 = step_at(lo, c, w), k1 = min(tiles, step_at(hi, c, w));
        if (k0 >= k1) return;
        u.valid = 1;
        u.nk = k1 - k0;
        u.key0 = k0 * kTile;
        u.tail = min(kTile, u.len - (k1 - 1) * kTile);
        segment(u);
      };

      int kind = sm.start[0], idx = sm.start[1], c = sm.start[2];
      Unit u;
      if (kind == 0) {
        for (; ok && c < hi && idx < p.num_groups; ++idx) {
          const Group g = load_group(p, idx);
          u.own = 0;
          u.len = g.len;
          u.table = p.prefix_table + static_cast<size_t>(idx) * p.max_prefix_pages;
          u.table_pages = p.max_prefix_pages;
          const int blocks = g.full + (g.rest > 0 ? 1 : 0);
          for (int blk = 0; ok && blk < blocks && g.tiles > 0; ++blk) {
            const int n = blk < g.full ? 2 * p.S : g.rest;
            u.both = n > p.S ? 1 : 0;
            const int w = u.both ? kCostBoth : kCostAlt;
            const int cost = job_cost(g.tiles, w);
            if (c + p.Hkv * cost <= lo) {  // wholly before this CTA's share
              c += p.Hkv * cost;
              continue;
            }
            u.b0 = g.b0 + blk * 2 * p.S;
            u.rows[0] = min(n, p.S) * p.G;
            u.rows[1] = u.both ? (n - p.S) * p.G : u.rows[0];
            for (int hk = 0; ok && hk < p.Hkv && c < hi; ++hk, c += cost) {
              u.hk = hk;
              u.out[0] = 2ll * p.G * p.Hkv * u.b0 + 2ll * p.G * n * hk +
                         static_cast<long long>(cta) * kCtaRows;
              u.out[1] = u.out[0] + u.rows[0];
              job(u, c, g.tiles, w);
            }
            if (c >= hi) break;
          }
        }
        if (ok && c < hi) {
          kind = 1;
          idx = 0;
        }
      }
      if (kind == 1) {
        u.own = 1;
        u.both = 0;
        u.rows[0] = u.rows[1] = p.G;
        u.table_pages = p.max_pages;
        for (; ok && c < hi && idx < p.B; ++idx) {
          u.len = seq_len(p, idx);
          const int tiles = (u.len + kTile - 1) / kTile;
          const int cost = job_cost(tiles, kCostAlt);
          u.b0 = idx;
          u.table = p.block_table + static_cast<size_t>(idx) * p.max_pages;
          for (int hk = 0; ok && tiles > 0 && hk < p.Hkv && c < hi; ++hk, c += cost) {
            u.hk = hk;
            u.out[0] = p.own_row0 + 2ll * p.G * (static_cast<long long>(idx) * p.Hkv + hk + cta);
            u.out[1] = u.out[0] + p.G;
            job(u, c, tiles, kCostAlt);
          }
        }
      }
      // the end: one segment that is not valid
      if (ok) {
        const int slot = published & 1;
        if (published >= 2)
          ok = wait_bounded(dev::smem_u32(&sm.bar_unit_empty[slot]), ((published - 2) >> 1) & 1, abort);
        if (lane == 0 && ok) {
          sm.unit[slot].valid = 0;
          __threadfence_block();
          dev::mbar_arrive(dev::smem_u32(&sm.bar_unit_full[slot]));
        }
      }
      __syncwarp();
      if (lane == 0) {
        // ---- drain: every copy this warp started has landed ----
        if (q_loads > 0) wait_drain(dev::smem_u32(&sm.bar_q), (q_loads - 1) & 1);
        for (int s = 0; s < 2; ++s) {
          // the last load into stage s among loads 0..n-1 completed phase (its number / 2)
          const int uk = (k_issued - 1 - s) >= 0 ? ((k_issued - 1 - s) & ~1) + s : -1;
          if (uk >= 0) wait_drain(dev::smem_u32(&sm.bar_kfull[s]), (uk >> 1) & 1);
          const int uv = (v_issued - 1 - s) >= 0 ? ((v_issued - 1 - s) & ~1) + s : -1;
          if (uv >= 0) wait_drain(dev::smem_u32(&sm.bar_vfull[s]), (uv >> 1) & 1);
        }
      }
    } else if (warp == kMmaWarp) {
      // ============================ tcgen05.mma issuer ============================
      // every lane walks the steps and waits; lane 0 issues
      constexpr uint32_t idesc_s = dev::idesc_bf16_f32(kTile, kTile, 0, 0);  // Q, K: K-major
      constexpr uint32_t idesc_o = dev::idesc_bf16_f32(kTile, kD, 0, 1);     // P (TMEM), V MN-major
      constexpr uint32_t kBufStep = kTileBytes >> 4;
      const uint64_t dq0 = dev::smem_desc(dev::smem_u32(sm.q[0]), 16, 1024, dev::kSwizzle128B);
      const uint64_t dk0 = dev::smem_desc(dev::smem_u32(sm.k[0]), 16, 1024, dev::kSwizzle128B);
      const uint64_t dv0 = dev::smem_desc(dev::smem_u32(sm.v[0]), kHalfBytes, 1024, dev::kSwizzle128B);
      bool ok = true;
      int taken = 0, q_waits = 0, gbase = 0;
      int ptot[2] = {0, 0};
      while (ok) {
        const int slot = taken & 1;
        ok = wait_bounded(dev::smem_u32(&sm.bar_unit_full[slot]), (taken >> 1) & 1, abort);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const Unit& us = sm.unit[slot];
        if (!us.valid) break;
        ++taken;
        const int nk = us.nk, both = us.both, flip = us.flip, tail = us.tail;
        int s_left = both ? 2 * nk : nk;  // S products of the segment still to issue
        // S of row tile t against the keys of step j; `last`: no other row tile reads them
        auto issue_s = [&](int t, int j, bool last) {
          const int g = gbase + j;
          bool w = wait_bounded(dev::smem_u32(&sm.bar_kfull[g & 1]), (g >> 1) & 1, abort);
          if (!(w = __all_sync(0xffffffffu, w))) return false;
          dev::tc_fence_after();
          if (lane == 0) {
            const uint64_t a0 = dq0 + static_cast<uint64_t>(both ? t * kBufStep : 0);
            const uint64_t b0 = dk0 + static_cast<uint64_t>((g & 1) * kBufStep);
#pragma unroll
            for (int ks = 0; ks < kD / 16; ++ks) {
              const uint32_t off = ((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
              dev::umma_ss(tmem + t * 128, a0 + off, b0 + off, idesc_s, ks > 0 ? 1u : 0u);
            }
            dev::umma_commit(dev::smem_u32(&sm.bar_s[t]));
            if (s_left == 1) dev::umma_commit(dev::smem_u32(&sm.bar_qempty));
            if (last) dev::umma_commit(dev::smem_u32(&sm.bar_kempty[g & 1]));
          }
          --s_left;
          __syncwarp();
          return true;
        };
        // O += P V of row tile t for step j
        auto issue_pv = [&](int t, int j, bool acc, bool last, bool final_step) {
          const int g = gbase + j;
          bool w = wait_bounded(dev::smem_u32(&sm.bar_p[t]), ptot[t] & 1, abort);
          if (!(w = __all_sync(0xffffffffu, w))) return false;
          ++ptot[t];
          dev::tc_fence_after();
          if (lane == 0) {
            const uint64_t b0 = dv0 + static_cast<uint64_t>((g & 1) * kBufStep);
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              dev::umma_ts(tmem + 256 + t * 128, tmem + t * 128 + ks * 8, b0 + ((ks * 16 * 128) >> 4),
                           idesc_o, (acc || ks > 0) ? 1u : 0u);
            if (last) dev::umma_commit(dev::smem_u32(&sm.bar_vempty[g & 1]));
            if (final_step) dev::umma_commit(dev::smem_u32(&sm.bar_o[t]));
          }
          __syncwarp();
          return true;
        };
        // the values of step j have landed; in the job's last tile the rows past the last key
        // become zeros
        auto wait_v = [&](int j) {
          const int g = gbase + j;
          bool w = wait_bounded(dev::smem_u32(&sm.bar_vfull[g & 1]), (g >> 1) & 1, abort);
          if (!(w = __all_sync(0xffffffffu, w))) return false;
          if (j == nk - 1 && tail < kTile) {
            const uint32_t base = dev::smem_u32(sm.v[g & 1]);
            for (uint32_t off = tail * 128u + lane * 16u; off < kHalfBytes; off += 512u) {
              dev::st_shared_v4(base + off, 0u, 0u, 0u, 0u);
              dev::st_shared_v4(base + kHalfBytes + off, 0u, 0u, 0u, 0u);
            }
            dev::fence_proxy_async_smem();
            __syncwarp();
          }
          return true;
        };
        ok = wait_bounded(dev::smem_u32(&sm.bar_q), q_waits & 1, abort);
        ok = __all_sync(0xffffffffu, ok);
        ++q_waits;
        if (both) {
          ok = ok && issue_s(0, 0, false) && issue_s(1, 0, true);
          for (int j = 0; ok && j < nk; ++j) {
            const bool more = j + 1 < nk;
            ok = wait_v(j) && issue_pv(0, j, j > 0, false, !more) && (!more || issue_s(0, j + 1, false)) &&
                 issue_pv(1, j, j > 0, true, !more) && (!more || issue_s(1, j + 1, true));
          }
        } else {
          ok = ok && issue_s(flip, 0, true) && (nk < 2 || issue_s(flip ^ 1, 1, true));
          for (int j = 0; ok && j < nk; ++j) {
            const int t = (j & 1) ^ flip;
            ok = wait_v(j) && issue_pv(t, j, j > 1, true, j + 2 >= nk) &&
                 (j + 2 >= nk || issue_s(t, j + 2, true));
          }
        }
        gbase += nk;
        if (lane == 0) dev::mbar_arrive(dev::smem_u32(&sm.bar_unit_empty[slot]));
      }
      __syncwarp();
      if (lane == 0) {
        dev::umma_commit(dev::smem_u32(&sm.bar_drain));
        wait_drain(dev::smem_u32(&sm.bar_drain), 0);
      }
    }
  } else {
    // ================ softmax + epilogue: one query row per thread ================
    dev::regs_increase<kRegsSoftmax>();
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_off + t * 128;
    const uint32_t t_o = tmem + lane_off + 256 + t * 128;
    const float masked = kNeg ? __int_as_float(0x7f800000) : neg_inf();
    const float c = p.c;
    bool ok = true;
    int taken = 0, stot = 0, otot = 0;
    while (ok) {
      const int slot = taken & 1;
      ok = wait_bounded(dev::smem_u32(&sm.bar_unit_full[slot]), (taken >> 1) & 1, abort);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const Unit& us = sm.unit[slot];
      if (!us.valid) break;
      ++taken;
      const int nk = us.nk, both = us.both, tail = us.tail;
      const int j0 = both ? 0 : t ^ us.flip;  // alt: the row tile's first step
      const int dj = both ? 1 : 2;
      const int rows = us.rows[t];
      const bool busy = (row & ~31) < rows;  // this warp has a real row
      float m_ref = neg_inf(), l = 0.f;
      int cnt = 0;
      for (int j = j0; j < nk; j += dj) {
        ok = wait_bounded(dev::smem_u32(&sm.bar_s[t]), stot & 1, abort);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        ++stot;
        if (busy) {
          dev::tc_fence_after();
          uint32_t r[128];
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) dev::tmem_ld32(t_s + cc * 32, r + cc * 32);
          dev::tmem_wait_ld_regs(r);
          if (j == nk - 1 && tail < kTile) {
#pragma unroll
            for (int e = 0; e < 128; ++e)
              r[e] = e < tail ? r[e] : __float_as_uint(masked);
          }
          float a[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = __uint_as_float(r[i]);
#pragma unroll
          for (int e = 8; e < 120; e += 16) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              a[i] = kNeg ? dev::min3(a[i], __uint_as_float(r[e + i]), __uint_as_float(r[e + 8 + i]))
                          : dev::max3(a[i], __uint_as_float(r[e + i]), __uint_as_float(r[e + 8 + i]));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            a[i] = kNeg ? fminf(a[i], __uint_as_float(r[120 + i])) : fmaxf(a[i], __uint_as_float(r[120 + i]));
          const float mx =
              kNeg ? dev::min3(dev::min3(a[0], a[1], a[2]), dev::min3(a[3], a[4], a[5]), fminf(a[6], a[7]))
                   : dev::max3(dev::max3(a[0], a[1], a[2]), dev::max3(a[3], a[4], a[5]), fmaxf(a[6], a[7]));
          const float tmax = mx == masked ? neg_inf() : mx * c;
          const float m_new = fmaxf(m_ref, tmax);
          float alpha = 1.f;
          if (m_new > m_ref + kRescaleThreshold) {
            alpha = dev::ex2_approx(m_ref - m_new);  // 0 from -inf
            m_ref = m_new;
          }
          l *= alpha;
          if (cnt > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // O *= alpha: the commit of S(j) covered this row tile's last P V
#pragma unroll 1
            for (int cc = 0; cc < 4; ++cc) {
              uint32_t o[32];
              dev::tmem_ld32(t_o + cc * 32, o);
              dev::tmem_wait_ld_regs(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              dev::tmem_st32(t_o + cc * 32, o);
            }
          }
          const float m_use = m_ref == neg_inf() ? 0.f : m_ref;
          const uint64_t c2 = dev::pack2(c, c), nm2 = dev::pack2(-m_use, -m_use);
          float2 acc[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              const int col = half * 64 + e;
              const float2 xx = dev::unpack2(dev::fma2(
                  dev::pack2(__uint_as_float(r[col]), __uint_as_float(r[col + 1])), c2, nm2));
              const float2 pr = make_float2(dev::ex2_approx(xx.x), dev::ex2_approx(xx.y));
              acc[(e >> 1) & 3] = dev::add2(acc[(e >> 1) & 3], pr);
              pk[e >> 1] = dev::pack_bf16x2(pr.x, pr.y);
            }
            dev::tmem_st32(t_s + half * 32, pk);
          }
          acc[0] = dev::add2(acc[0], acc[1]);
          acc[2] = dev::add2(acc[2], acc[3]);
          acc[0] = dev::add2(acc[0], acc[2]);
          l += acc[0].x + acc[0].y;
          dev::tmem_wait_st();
          dev::tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(dev::smem_u32(&sm.bar_p[t]));
        ++cnt;
      }
      // ---- epilogue: O / l and its log-sum-exp, as partial rows ----
      if (cnt > 0 && ok) ok = wait_bounded(dev::smem_u32(&sm.bar_o[t]), otot & 1, abort);
      if (cnt > 0) ++otot;
      ok = __all_sync(0xffffffffu, ok);
      if (ok && cnt > 0 && busy) {
        dev::tc_fence_after();
        // alt mode: the row tile that took the first step writes the first rows
        const long long out0 = us.out[both ? t : t ^ us.flip] + (row & ~31);
        const int live = min(32, rows - (row & ~31));  // real rows of this warp
        const float inv_l = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        const uint32_t box = dev::smem_u32(sm.stage[warp]);
#pragma unroll 1
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t o[32];
          dev::tmem_ld32(t_o + cc * 32, o);
          dev::tmem_wait_ld_regs(o);
          // 16-byte chunk i of row r at chunk i ^ (r & 7): no bank conflicts either way
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dev::st_shared_v4(box + lane * 128 + ((i ^ (lane & 7)) << 4),
                              __float_as_uint(__uint_as_float(o[4 * i]) * inv_l),
                              __float_as_uint(__uint_as_float(o[4 * i + 1]) * inv_l),
                              __float_as_uint(__uint_as_float(o[4 * i + 2]) * inv_l),
                              __float_as_uint(__uint_as_float(o[4 * i + 3]) * inv_l));
          __syncwarp();
#pragma unroll 1
          for (int r0 = 0; r0 < live; r0 += 4) {
            const int r = r0 + (lane >> 3), i = lane & 7;
            if (r < live) {
              const uint4 x = *reinterpret_cast<const uint4*>(sm.stage[warp] + r * 128 + ((i ^ (r & 7)) << 4));
              *reinterpret_cast<uint4*>(p.ws_o + (out0 + r) * kD + cc * 32 + i * 4) = x;
            }
          }
          __syncwarp();
        }
        if (lane < live) {
          const float m_use = m_ref == neg_inf() ? 0.f : m_ref;
          p.ws_lse[out0 + lane] = l == 0.f ? neg_inf() : (m_use + log2f(l)) * 0.69314718055994531f;
        }
      }
      dev::tc_fence_before();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(dev::smem_u32(&sm.bar_unit_empty[slot]));
    }
  }

  // ---- teardown ----
  dev::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    dev::tc_fence_after();
    dev::tmem_dealloc(tmem, 512);
  }
}

// Join the parts of one query row: one warp per (sequence, query head), four columns a lane.
constexpr int kCombineWarps = 8;

// The parts of a row, numbered in line order: those of the prefix job, then those of the own job.
struct Parts {
  int c, w, tiles;  // the job: position on the line, weight and number of its steps (0: none)
  int first, ctas;  // CTAs that hold a part of it
  int both;
  long long row;    // the query row's first partial row as held by CTA 0
  int cta_rows;     // rows from one CTA's part to the next one's
  int alt_rows;     // alt mode: rows from the even steps' part to the odd steps' part
};

__global__ void __launch_bounds__(kCombineWarps * 32)
    decode_prefix_combine_kernel(const Params p, __nv_bfloat16* __restrict__ o,
                                 float* __restrict__ lse) {
  const int lane = threadIdx.x & 31;
  const long long bh = static_cast<long long>(blockIdx.x) * kCombineWarps + (threadIdx.x >> 5);
  if (bh >= static_cast<long long>(p.B) * p.Hq) return;
  const int b = static_cast<int>(bh / p.Hq), h = static_cast<int>(bh % p.Hq);
  const int hk = h / p.G, gq = h % p.G;
  const int share = p.plan[0];

  Parts part[2];
  part[0].tiles = part[0].ctas = 0;
  part[1].tiles = part[1].ctas = 0;
  // the group of the sequence: the last one that starts at or before it
  int g = -1;
  if (p.num_groups > 0) {
    int a = 0, e = p.num_groups;  // starts[a] <= b < starts[e]
    if (__ldg(p.group_starts) <= b) {
      while (e - a > 1) {
        const int m = (a + e) >> 1;
        if (__ldg(p.group_starts + m) <= b) a = m;
        else e = m;
      }
      g = a;
    }
  }
  if (g >= 0) {
    const Group gr = load_group(p, g);
    if (b < gr.b0 + gr.n && gr.tiles > 0) {
      const int blk = (b - gr.b0) / (2 * p.S), in = (b - gr.b0) % (2 * p.S);
      const int n = blk < gr.full ? 2 * p.S : gr.rest;
      Parts& x = part[0];
      x.both = n > p.S ? 1 : 0;
      x.w = x.both ? kCostBoth : kCostAlt;
      x.tiles = gr.tiles;
      x.c = p.plan[2 + g] + p.Hkv * blk * job_cost(gr.tiles, kCostBoth) + hk * job_cost(gr.tiles, x.w);
      x.row = 2ll * p.G * p.Hkv * (gr.b0 + blk * 2 * p.S) + 2ll * p.G * n * hk + in * p.G + gq;
      x.cta_rows = kCtaRows;
      x.alt_rows = n * p.G;
    }
  }
  const int own_len = seq_len(p, b);
  if (own_len > 0) {
    Parts& x = part[1];
    x.both = 0;
    x.w = kCostAlt;
    x.tiles = (own_len + kTile - 1) / kTile;
    x.c = p.plan[2 + p.num_groups + b] + hk * job_cost(x.tiles, kCostAlt);
    x.row = p.own_row0 + 2ll * p.G * (static_cast<long long>(b) * p.Hkv + hk) + gq;
    x.cta_rows = 2 * p.G;
    x.alt_rows = p.G;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    Parts& x = part[i];
    if (x.tiles > 0) {
      x.first = x.c / share;
      x.ctas = (x.c + (x.tiles - 1) * x.w) / share - x.first + 1;
    }
  }
  // part number e of a job: CTA first + e / 2, even or odd steps; -1 where it holds nothing
  const int n0 = 2 * part[0].ctas, n1 = 2 * part[1].ctas;
  auto row_of = [&](int e) -> long long {
    const Parts& x = e < n0 ? part[0] : part[1];
    if (e >= n0) e -= n0;
    const int cta = x.first + (e >> 1);
    if (e & 1) {
      // the odd steps' part exists in alt mode if the CTA holds two steps or more
      if (x.both) return -1;
      const int k0 = step_at(cta * share, x.c, x.w);
      const long long next = static_cast<long long>(cta + 1) * share;
      const int end = next > 0x7fffffff ? 0x7fffffff : static_cast<int>(next);
      const int k1 = min(x.tiles, step_at(end, x.c, x.w));
      if (k1 - k0 < 2) return -1;
    }
    return x.row + static_cast<long long>(cta) * x.cta_rows + ((e & 1) ? x.alt_rows : 0);
  };
  float top = neg_inf(), z = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  // 32 parts at a time: a lane reads one part's log-sum-exp, then the warp adds the parts up
  for (int e0 = 0; e0 < n0 + n1; e0 += 32) {
    long long row = -1;
    float L = neg_inf();
    if (e0 + lane < n0 + n1) row = row_of(e0 + lane);
    if (row >= 0) L = p.ws_lse[row];
    float mx = L;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    const float new_top = fmaxf(top, mx);
    const float f = new_top == neg_inf() ? 1.f : expf(top - new_top);
    z *= f;
    acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
    top = new_top;
    // a NaN part (NaN inputs) keeps its NaN
    const float wgt = L == neg_inf() ? 0.f : expf(L - top);
    unsigned live = __ballot_sync(0xffffffffu, row >= 0 && !(wgt == 0.f));
    while (live) {
      const int src = __ffs(live) - 1;
      live &= live - 1;
      const float w = __shfl_sync(0xffffffffu, wgt, src);
      const long long rw = __shfl_sync(0xffffffffu, row, src);
      const float4 x = *reinterpret_cast<const float4*>(p.ws_o + rw * kD + 4 * lane);
      z += w;
      acc.x = fmaf(w, x.x, acc.x);
      acc.y = fmaf(w, x.y, acc.y);
      acc.z = fmaf(w, x.z, acc.z);
      acc.w = fmaf(w, x.w, acc.w);
    }
  }
  const float inv = z == 0.f ? 0.f : 1.f / z;
  uint2 out;
  out.x = dev::pack_bf16x2(acc.x * inv, acc.y * inv);
  out.y = dev::pack_bf16x2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(o + bh * kD + 4 * lane) = out;
  if (lane == 0 && lse != nullptr) lse[bh] = z == 0.f ? neg_inf() : top + logf(z);
}

}  // namespace pfx
}  // namespace attn
