// Decode for a batch whose sequences share long prefixes, over a paged KV cache: the keys of a
// prefix are read once for all the sequences behind it, those of a sequence's own pages once for
// that sequence, and the parts are joined exactly by their log-sum-exps.
//
// The mathematics is that of decode.cuh: with the keys of one query row split into parts, part s
// gives O_s = sum_j 2^(x_j - m_s) v_j / l_s and lse_s = ln(sum exp); then LSE = ln sum_s
// exp(lse_s) and O = sum_s exp(lse_s - LSE) O_s.
//
// Scores, running maxima, sums, the parts and their log-sum-exps are fp32.  The weights are rounded to bf16 (half a
// step, 2^-8 of a weight at most), because both operands of a tensor-core product have one type and V is
// bf16; the sums l take them before that rounding.  Weights in two bf16 terms would keep fp32's bits, and double the
// products with V and the stores of P in the wide steps, which computing bounds.  O comes out with 0.0023 of relative
// error where its own rounding to bf16 costs 0.0017; LSE is not touched.
//
// Work.  A job is one kv head of either a block of sequences of one group (their query rows
// against the prefix keys) or one sequence (its G query rows against its own keys); a step is one
// 128-key tile of a job.  How a step is computed depends on the query rows of its job:
//   both  more than 128 rows (at most 256): S = Q K^T with the rows as M, P from tensor memory for
//         O += P V; two row tiles take every step, so a key tile read once feeds up to 256 rows.
//         2.4 us a step with every SM at it (4.0 TB/s of keys and values): scores, softmax of 32768
//         weights and P V follow each other in each row tile, and the two row tiles overlap only in part.
//   alt   17 to 128 rows: the same with the two row tiles holding the same rows and taking
//         alternate steps, so one step's softmax overlaps the next step's products; even and odd
//         steps end as two parts.  1.55 us a step with every SM at it, 6.2 TB/s.
//   thin  at most 16 rows (every sequence's own keys among them): S^T = K Q^T with the keys as M and
//         16 columns, O^T += V^T P^T; a thread holds a key's few scores, so a step costs far
//         less than its 64 KB take to arrive.
// The steps of 256 rows are bound by computing, the others by HBM where all SMs take them, and they run beside
// each other on different SMs: the steps of each kind stand in a line, weighted by what they cost,
// the CTAs (persistent, one per SM) are divided between the two lines, and every CTA takes an equal
// length of its line.  Long prefixes are so cut over many CTAs, short sequences taken several to a
// CTA.  The cuts follow from the lengths alone, which each CTA sums up for itself when it
// starts: there is no counter and no order of arrival, results are the same in every run, and
// launches share nothing but the caller's workspace.
//
// Measured on a B200 (Hq 32, Hkv 8; both kernels): 64 sequences behind 32768 keys, 400 own at most, 16-key
// pages: 71.3 us; 256 sequences behind 16384 keys, 1500 own at most, 32-key pages: 201 us (218-228 where calls
// follow each other for long, under the power cap at 1.75 GHz); 4 behind 700 keys: 15.7 us.  Own keys alone
// (64 x 4096 keys): 5.9 TB/s with 16-key pages, 6.3 with 64.  What a call takes beside its steps (launch, plan,
// first loads, epilogues, the joining kernel): 14.3, 16.9 and 18.7 us around a single tile for 16, 128 and 256 rows;
// 19, 23 and 25 us where every job is cut over many CTAs (64-key pages, a line through 18944 to 75776 keys).
//
// Warps (12): 0-3 and 4-7 softmax and epilogue (wide: of row tile 0 and 1, thread = row = TMEM lane;
// thin: of even and odd chunks of 4 tiles, thread = key, then output column), 8 the tcgen05.mma
// issuer (all lanes first zero the value rows past a job's last key: what a page holds there may
// be infinite or NaN, and 0 x NaN would reach the sum), 9 the job walk and the TMA producer (one
// lane per box: a 128-key tile is 128 / min(page size, 128) pieces), 10-11 idle.
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
constexpr uint32_t kHalfBytes = kTile * 64 * 2;  // a query row tile: column half after column half
// A key or value tile: 8 rows of the first column half, the same 8 rows of the second (128-byte rows,
// 128-byte swizzle), then the next 8 rows.  So a piece of a page is one box of a 5-D tensor map, both
// halves in it: a box costs the TMA unit about 50 clocks on top of 64 bytes a clock, and with
// 16-key pages an SM takes in 32 bytes a clock instead of 23 with a box per half (80 SMs: 25, 19).
constexpr uint32_t kGroupBytes = 2048, kGroupHalf = 1024;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

// Costs on the lines, in units of about 245 SM clocks: a step of each kind, and what a job adds (its
// first products and its epilogue, which overlap other jobs' only in part; charged once a job, though each
// CTA that the job is cut over has its own).  A thin step takes what
// its 64 KB take through the TMA unit, which depends on the size of the boxes, so of the pages
// (page_shift 3, 4, 5, 6 and more: 17, 25, 36 and 40 bytes a clock with 80 SMs at it).
constexpr int kCostBoth = 16;
constexpr int kCostAlt = 10;
constexpr int kCostWideJob = 24;
constexpr int kCostThinJob = 3;
__host__ __device__ constexpr int cost_thin_step(int page_shift) {
  return page_shift <= 3 ? 15 : page_shift == 4 ? 10 : page_shift == 5 ? 8 : 7;
}
constexpr int kCostThinMax = 15;
// HBM takes 19 clocks for the 64 KB of a step: 5 / 64 units
constexpr int kHbmNum = 5, kHbmDen = 64;

constexpr int kThinRows = 16;   // query rows of a thin job
constexpr int kChunk = 4;       // tiles of a thin chunk
constexpr int kThinStages = 5;  // tiles on their way in a thin CTA
// The values of a CTA's last chunk are all streamed before the end is published, and the tensor core
// takes them after it has seen the end: the ring has to hold them.  (4 and 5 stages measure alike.)
static_assert(kThinStages >= kChunk, "the last chunk's values wait in the ring");

// Rows of partial results, by region: a job's rows start at 2 G Hkv (its first sequence) + 2 G n (its kv
// head) for a block of n sequences, and every CTA adds its index times a stride that is not below
// what a segment holds (256, 32 and 2 G rows): segments in line order never overlap.
constexpr int kWideCtaRows = 256;
constexpr int kThinCtaRows = 2 * kThinRows;

struct Params {
  int B, Hq, Hkv, G, S;  // S = 128 / G: sequences in one row tile
  int num_groups, max_prefix_len, max_prefix_pages;
  int max_seq_len, max_pages;
  int num_pages, page_shift, thin_cost;  // thin_cost: cost_thin_step(page_shift)
  const int* prefix_table;  // [num_groups][max_prefix_pages]
  const int* prefix_lens;   // [num_groups]
  const int* group_starts;  // [num_groups + 1]
  const int* block_table;   // [B][max_pages]
  const int* seq_lens;      // [B]
  float c;                  // scale * log2(e), never 0
  float* ws_o;              // partial outputs [rows][128], then
  float* ws_lse;            // their log-sum-exps [rows]
  int* plan;                // [0] share of a wide CTA, [1] of a thin CTA, [2] wide CTAs, [3] whether the
                            // prefixes count (the groups are in order), then positions on the lines: of each group's wide jobs [num_groups], of its
                            // thin jobs [num_groups], of each sequence's own jobs [B]
  long long thin_row0, own_row0;  // first rows of the thin prefix parts and of the own parts
};

// ---- the lines of jobs (shared with the combine kernel) ----
struct Group {
  int b0 = 0, n = 0, tiles = 0, len = 0;  // first sequence, sequences, key tiles, keys
  int full = 0, rest = 0;                 // blocks of 2 S sequences, sequences of the last, smaller block
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return max(lo, min(x, hi)); }

__device__ __forceinline__ Group load_group(const Params& p, int g) {
  Group r;
  const int a = __ldg(p.group_starts + g), e = __ldg(p.group_starts + g + 1), len = __ldg(p.prefix_lens + g);
  r.b0 = clampi(a, 0, p.B);
  r.n = clampi(e, r.b0, p.B) - r.b0;
  r.len = clampi(len, 0, p.max_prefix_len);
  r.tiles = (r.len + kTile - 1) / kTile;
  r.full = r.n / (2 * p.S);
  r.rest = r.n % (2 * p.S);
  return r;
}
__device__ __forceinline__ bool rest_thin(const Params& p, const Group& g) { return g.rest * p.G <= kThinRows; }
__device__ __forceinline__ int wide_weight(const Params& p, int n) { return n > p.S ? kCostBoth : kCostAlt; }
__device__ __forceinline__ int wide_job(int tiles, int weight) { return tiles > 0 ? tiles * weight + kCostWideJob : 0; }
__device__ __forceinline__ int thin_job(const Params& p, int tiles) {
  return tiles > 0 ? tiles * p.thin_cost + kCostThinJob : 0;
}
// a group's jobs on the wide line and on the thin line
__device__ __forceinline__ int group_wide(const Params& p, const Group& g) {
  const int rest = g.rest > 0 && !rest_thin(p, g) ? wide_job(g.tiles, wide_weight(p, g.rest)) : 0;
  return p.Hkv * (g.full * wide_job(g.tiles, kCostBoth) + rest);
}
__device__ __forceinline__ int group_thin(const Params& p, const Group& g) {
  return g.rest > 0 && rest_thin(p, g) ? p.Hkv * thin_job(p, g.tiles) : 0;
}
__device__ __forceinline__ int seq_len(const Params& p, int b) {
  return clampi(__ldg(p.seq_lens + b), 0, p.max_seq_len);
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }
// first step at or after position x of a line, for a job at position c with steps of weight w
__device__ __forceinline__ int step_at(int x, int c, int w) { return x <= c ? 0 : (x - c + w - 1) / w; }

// A run of steps of one wide job.
struct Unit {
  int valid;
  int both;          // 1: both row tiles take every step; 0: alternate steps
  int flip;          // alt mode: the row tile that takes the first step
  int nk;            // steps
  int tail;          // keys of the last step (1..128)
  int rows[2];       // real query rows of each row tile
  long long out[2];  // first partial row of each row tile
  int b0, hk;        // first sequence, kv head
};

// At most kChunk steps of one thin job.
struct Chunk {
  int valid;
  int nt, keys;     // tiles, keys
  int cols;         // query rows (columns of S^T)
  int first, last;  // first / last chunk of its segment that its softmax group takes
  int only;         // the segment has no other chunk
  long long out;    // partial rows of its softmax group
};
constexpr int kChunkSlots = 4;
constexpr uint32_t kQHalfBytes = kThinRows * 128;
constexpr uint32_t kPBlockBytes = kThinRows * 128;  // P^T rows of 64 keys
constexpr uint32_t kPTileBytes = 2 * kPBlockBytes;

struct WideSmem {
  uint8_t q[2][kTileBytes];
  uint8_t k[2][kTileBytes];
  uint8_t v[2][kTileBytes];
};
struct ThinSmem {
  uint8_t tile[kThinStages][kTileBytes];
  uint8_t q[kThinStages][2 * kQHalfBytes];  // every key tile comes with its own copy of the queries
  uint8_t p[2][kChunk][kPTileBytes];
};
struct __align__(1024) Smem {
  union {
    WideSmem w;
    ThinSmem t;
  };
  // wide
  uint64_t bar_q, bar_qempty;
  uint64_t bar_kfull[2], bar_kempty[2], bar_vfull[2], bar_vempty[2];
  uint64_t bar_unit_full[2], bar_unit_empty[2];
  // thin
  uint64_t bar_full[kThinStages], bar_empty[kThinStages];
  uint64_t bar_chunk_full[kChunkSlots], bar_chunk_empty[kChunkSlots];
  // both
  uint64_t bar_s[2], bar_p[2], bar_o[2], bar_group[2], bar_drain;
  Unit unit[2];
  Chunk chunk[kChunkSlots];
  float red[2][2][2][4][kThinRows];  // per softmax group: its warps' maxima and sums, two buffers each
  int4 scan[kThreads / 32];
  int start[3];  // where this CTA's share begins: kind, group or sequence, position of its first job
  uint32_t tmem_base;
  int abort;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");
constexpr uint32_t kUnitReaders = 9;   // 8 softmax warps, the MMA warp
constexpr uint32_t kChunkReaders = 5;  // 4 softmax warps of its group, the MMA warp

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// What the roles of a CTA share.
struct Cta {
  Smem* sm;
  uint32_t tmem;
  int index;   // among the CTAs of its line
  int lo, hi;  // its share of the line
};

// A sequence's own keys are read once and leave L2 first (64 sequences of 4096 keys: 5.74 -> 5.84 TB/s with 16-key
// pages, 6.16 -> 6.36 with 64; 97 sequences in 5 groups 48.5 -> 47.1 us; to hold a prefix's keys back from
// leaving, beyond that, changes nothing).
__device__ __forceinline__ uint64_t prefix_policy() {
  uint64_t x;
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(x));
  return x;
}
__device__ __forceinline__ uint64_t own_policy() {
  uint64_t x;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(x));
  return x;
}

// One box: `piece` rows of one kv head, both column halves; row0 is a multiple of 8.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int row0, int hk,
                                         uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %3, %3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(row0 >> 3), "r"(hk), "l"(policy)
      : "memory");
}

// The piece of a tile that this lane of the producer warp loads.
struct Pieces {
  int psize, piece, pieces, mine;
  int rows_total;
  __device__ __forceinline__ explicit Pieces(const Params& p) {
    psize = 1 << p.page_shift;
    piece = psize < kTile ? psize : kTile;
    pieces = kTile / piece;
    mine = threadIdx.x & 31;
    rows_total = static_cast<int>(static_cast<long long>(p.num_pages) << p.page_shift);
  }
  // page of this lane's piece of the tile at key0, -2 if it holds no key below len
  __device__ __forceinline__ int page(const Params& p, const int* table, int table_pages, int key0, int len) const {
    const int key = key0 + mine * piece;
    if (mine >= pieces || key >= len) return -2;
    const int lp = key >> p.page_shift;
    return lp < table_pages ? __ldg(table + lp) : -1;
  }
  // its row of the page pool; a page outside the cache is not followed: past the last row, reads as zero
  __device__ __forceinline__ int row(const Params& p, int page, int key0) const {
    if (page >= 0 && page < p.num_pages) return (page << p.page_shift) + ((key0 + mine * piece) & (psize - 1));
    if (page != -2) atomicExch(&g_device_error, ATTN_ERR_INVALID_ARG);
    return rows_total;
  }
  __device__ __forceinline__ uint32_t bytes(int key0, int len) const {
    return static_cast<uint32_t>(min(pieces, (len - key0 + piece - 1) / piece)) * piece * 256u;
  }
  __device__ __forceinline__ void load(const CUtensorMap* map, uint32_t dst, uint32_t bar, int page, int row, int hk,
                                       uint64_t policy) const {
    if (page != -2) load_box(dst + mine * piece * 256, map, bar, row, hk, policy);
  }
};

// wait of a whole warp
__device__ __forceinline__ bool warp_wait(uint64_t* bar, int phase, volatile int* abort) {
  const bool ok = wait_bounded(dev::smem_u32(bar), phase & 1, abort);
  return __all_sync(0xffffffffu, ok);
}

// value rows tail.. of a landed tile become zeros (a whole warp), visible to the tensor core
__device__ __forceinline__ void zero_tail(uint32_t tile, int tail) {
  for (int i = threadIdx.x & 31; i < (kTile - tail) * 16; i += 32) {
    const uint32_t row = tail + (i >> 4), half = (i >> 3) & 1, chunk = i & 7;
    dev::st_shared_v4(tile + (row >> 3) * kGroupBytes + half * kGroupHalf + (row & 7) * 128 + chunk * 16, 0u, 0u, 0u, 0u);
  }
  dev::fence_proxy_async_smem();
  __syncwarp();
}

// ------------------------------------------------------------------------------------------
// wide CTAs
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ void wide_produce(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                             const CUtensorMap& tm_v, const Params& p, const Cta& ct) {
  Smem& sm = *ct.sm;
  const int lane = threadIdx.x & 31;
  volatile int* abort = &sm.abort;
  const Pieces pc(p);
  const uint64_t policy = prefix_policy();
  int published = 0, q_loads = 0, k_issued = 0, v_issued = 0;
  bool ok = true;

  // publish one run of steps and stream its tiles
  auto run = [&](Unit& u, int key0, int len, const int* table) {
    const int slot = published & 1;
    if (published >= 2 && !(ok = warp_wait(&sm.bar_unit_empty[slot], (published - 2) >> 1, abort))) return;
    u.flip = u.both ? 0 : published & 1;
    if (lane == 0) {
      sm.unit[slot] = u;
      __threadfence_block();
      dev::mbar_arrive(dev::smem_u32(&sm.bar_unit_full[slot]));
    }
    __syncwarp();
    ++published;
    // Q once the previous run's last S products have read the Q buffers
    if (q_loads > 0 && !(ok = warp_wait(&sm.bar_qempty, q_loads - 1, abort))) return;
    if (lane == 0) {
      const uint32_t bq = dev::smem_u32(&sm.bar_q);
      const int tiles = u.both ? 2 : 1;
      dev::mbar_arrive_expect_tx(bq, tiles * kTileBytes);
      for (int t = 0; t < tiles; ++t)
        for (int half = 0; half < 2; ++half)
          dev::tma_load_3d(dev::smem_u32(sm.w.q[t]) + half * kHalfBytes, &tm_q, bq, half * 64, u.hk * p.G,
                           u.b0 + t * p.S);
    }
    __syncwarp();
    ++q_loads;
    // Keys of step j, then its values; in alt mode the keys run a step ahead, because S does.
    auto load = [&](bool keys, int page, int j) {
      int& count = keys ? k_issued : v_issued;
      const int s = count & 1, ph = (count >> 1) ^ 1, at = key0 + j * kTile;
      const int row = pc.row(p, page, at);
      if (!(ok = warp_wait(keys ? &sm.bar_kempty[s] : &sm.bar_vempty[s], ph, abort))) return false;
      const uint32_t bar = dev::smem_u32(keys ? &sm.bar_kfull[s] : &sm.bar_vfull[s]);
      if (lane == 0) dev::mbar_arrive_expect_tx(bar, pc.bytes(at, len));
      __syncwarp();
      pc.load(keys ? &tm_k : &tm_v, dev::smem_u32(keys ? sm.w.k[s] : sm.w.v[s]), bar, page, row, u.hk, policy);
      ++count;
      return true;
    };
    auto page_of = [&](int j) {
      return j < u.nk ? pc.page(p, table, p.max_prefix_pages, key0 + j * kTile, len) : -2;
    };
    int page = page_of(0), next = page_of(1);
    if (!load(true, page, 0)) return;
    for (int j = 0; j < u.nk; ++j) {
      const int cur = page;
      page = next;
      next = page_of(j + 2);
      if (u.both && !load(false, cur, j)) return;
      if (j + 1 < u.nk && !load(true, page, j + 1)) return;
      if (!u.both && !load(false, cur, j)) return;
    }
  };

  if (sm.start[0] == 0) {
    int c = sm.start[2];
    Unit u;
    u.valid = 1;
    for (int idx = sm.start[1]; ok && c < ct.hi && idx < p.num_groups; ++idx) {
      const Group g = load_group(p, idx);
      const int* table = p.prefix_table + static_cast<size_t>(idx) * p.max_prefix_pages;
      const int blocks = g.tiles == 0 ? 0 : g.full + (g.rest > 0 && !rest_thin(p, g) ? 1 : 0);
      for (int blk = 0; ok && c < ct.hi && blk < blocks; ++blk) {
        const int n = blk < g.full ? 2 * p.S : g.rest;
        const int w = wide_weight(p, n), cost = wide_job(g.tiles, w);
        if (c + p.Hkv * cost <= ct.lo) {  // wholly before this CTA's share
          c += p.Hkv * cost;
          continue;
        }
        u.both = n > p.S ? 1 : 0;
        u.b0 = g.b0 + blk * 2 * p.S;
        u.rows[0] = min(n, p.S) * p.G;
        u.rows[1] = u.both ? (n - p.S) * p.G : u.rows[0];
        for (int hk = 0; ok && c < ct.hi && hk < p.Hkv; ++hk, c += cost) {
          const int k0 = step_at(ct.lo, c, w), k1 = min(g.tiles, step_at(ct.hi, c, w));
          if (k0 >= k1) continue;
          u.hk = hk;
          u.out[0] = 2ll * p.G * p.Hkv * u.b0 + 2ll * p.G * n * hk + static_cast<long long>(ct.index) * kWideCtaRows;
          u.out[1] = u.out[0] + u.rows[0];
          u.nk = k1 - k0;
          u.tail = min(kTile, g.len - (k1 - 1) * kTile);
          run(u, k0 * kTile, g.len, table);
        }
      }
    }
  }
  // the end: a run that is not valid
  if (ok) {
    const int slot = published & 1;
    if (published >= 2) ok = warp_wait(&sm.bar_unit_empty[slot], (published - 2) >> 1, abort);
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
}

// every lane walks the steps and waits; lane 0 issues
__device__ __forceinline__ void wide_mma(const Cta& ct) {
  Smem& sm = *ct.sm;
  const int lane = threadIdx.x & 31;
  const uint32_t tmem = ct.tmem;
  volatile int* abort = &sm.abort;
  constexpr uint32_t idesc_s = dev::idesc_bf16_f32(kTile, kTile, 0, 0);  // Q, K: K-major
  constexpr uint32_t idesc_o = dev::idesc_bf16_f32(kTile, kD, 0, 1);     // P (TMEM), V MN-major
  constexpr uint32_t kBufStep = kTileBytes >> 4;
  const uint64_t dq0 = dev::smem_desc(dev::smem_u32(sm.w.q[0]), 16, 1024, dev::kSwizzle128B);
  const uint64_t dk0 = dev::smem_desc(dev::smem_u32(sm.w.k[0]), 16, kGroupBytes, dev::kSwizzle128B);
  const uint64_t dv0 = dev::smem_desc(dev::smem_u32(sm.w.v[0]), kGroupHalf, kGroupBytes, dev::kSwizzle128B);
  bool ok = true;
  int taken = 0, gbase = 0;
  int ptot0 = 0, ptot1 = 0;
  while (ok) {
    const int slot = taken & 1;
    if (!(ok = warp_wait(&sm.bar_unit_full[slot], taken >> 1, abort))) break;
    const Unit& us = sm.unit[slot];
    if (!us.valid) break;
    ++taken;
    const int nk = us.nk, both = us.both, flip = us.flip, tail = us.tail;
    // Item x of the run: row tile and step.  S runs two items ahead of P V.
    const int items = both ? 2 * nk : nk;
    auto tile_of = [&](int x) { return (x & 1) ^ flip; };
    auto step_of = [&](int x) { return both ? x >> 1 : x; };
    ok = warp_wait(&sm.bar_q, taken - 1, abort);
#pragma unroll 1
    for (int x = 0; ok && x < items + 2; ++x) {
      if (x >= 2) {
        // O += P V, once the values have landed; behind the job's last key they become zeros
        const int t = tile_of(x), j = step_of(x - 2), g = gbase + j;
        if (!both || t == 0) {
          if (!(ok = warp_wait(&sm.bar_vfull[g & 1], g >> 1, abort))) break;
          if (j == nk - 1 && tail < kTile) zero_tail(dev::smem_u32(sm.w.v[g & 1]), tail);
        }
        if (!(ok = warp_wait(&sm.bar_p[t], t ? ptot1 : ptot0, abort))) break;
        if (t) ++ptot1;
        else ++ptot0;
        dev::tc_fence_after();
        if (lane == 0) {
          const uint64_t b0 = dv0 + static_cast<uint64_t>((g & 1) * kBufStep);
          const bool acc = both ? j > 0 : j > 1;
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            dev::umma_ts(tmem + 256 + t * 128, tmem + t * 128 + ks * 8, b0 + ((ks * 2 * kGroupBytes) >> 4), idesc_o,
                         (acc || ks > 0) ? 1u : 0u);
          if (!both || t == 1) dev::umma_commit(dev::smem_u32(&sm.bar_vempty[g & 1]));
          if (x >= items) dev::umma_commit(dev::smem_u32(&sm.bar_o[t]));  // the row tile's last
        }
        __syncwarp();
      }
      if (x < items) {
        const int t = tile_of(x), g = gbase + step_of(x);
        if (!(ok = warp_wait(&sm.bar_kfull[g & 1], g >> 1, abort))) break;
        dev::tc_fence_after();
        if (lane == 0) {
          const uint64_t a0 = dq0 + static_cast<uint64_t>(both ? t * kBufStep : 0);
          const uint64_t b0 = dk0 + static_cast<uint64_t>((g & 1) * kBufStep);
#pragma unroll
          for (int ks = 0; ks < kD / 16; ++ks) {
            const uint32_t qoff = ((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
            const uint32_t koff = ((ks >> 2) * kGroupHalf + (ks & 3) * 32) >> 4;
            dev::umma_ss(tmem + t * 128, a0 + qoff, b0 + koff, idesc_s, ks > 0 ? 1u : 0u);
          }
          dev::umma_commit(dev::smem_u32(&sm.bar_s[t]));
          if (x == items - 1) dev::umma_commit(dev::smem_u32(&sm.bar_qempty));
          if (!both || t == 1) dev::umma_commit(dev::smem_u32(&sm.bar_kempty[g & 1]));
        }
        __syncwarp();
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

// Softmax and epilogue of one row tile, one query row per thread.
template <bool kNeg>
__device__ __forceinline__ void wide_softmax(const Params& p, const Cta& ct) {
  Smem& sm = *ct.sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = warp >> 2, row = tid & 127;
  volatile int* abort = &sm.abort;
  const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t t_s = ct.tmem + lane_off + t * 128;
  const uint32_t t_o = ct.tmem + lane_off + 256 + t * 128;
  const float masked = kNeg ? __int_as_float(0x7f800000) : neg_inf();
  const float c = p.c;
  bool ok = true;
  int taken = 0, stot = 0, otot = 0;
  while (ok) {
    const int slot = taken & 1;
    if (!(ok = warp_wait(&sm.bar_unit_full[slot], taken >> 1, abort))) break;
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
      if (!(ok = warp_wait(&sm.bar_s[t], stot, abort))) break;
      ++stot;
      if (busy) {
        dev::tc_fence_after();
        uint32_t r[128];
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) dev::tmem_ld32(t_s + cc * 32, r + cc * 32);
        dev::tmem_wait_ld_regs(r);
        if (j == nk - 1 && tail < kTile) {
#pragma unroll
          for (int e = 0; e < 128; ++e) r[e] = e < tail ? r[e] : __float_as_uint(masked);
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
    // (alt mode with a single step: this row tile's half of the part holds nothing)
    if (ok && cnt == 0 && row < rows) p.ws_lse[us.out[t ^ us.flip] + row] = neg_inf();
    // ---- epilogue: O / l and its log-sum-exp, as partial rows ----
    if (cnt > 0 && ok) {
      ok = warp_wait(&sm.bar_o[t], otot, abort);
      ++otot;
    }
    if (ok && cnt > 0 && busy) {
      dev::tc_fence_after();
      // alt mode: the row tile that took the first step writes the first rows.  A part's rows lie 16
      // bytes of every row after 16 bytes of every row, so a warp's store is 512 bytes in one run.
      const long long out = us.out[both ? t : t ^ us.flip];
      const bool real = row < rows;
      const float inv_l = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      uint4* dst = reinterpret_cast<uint4*>(p.ws_o + out * kD) + row;
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t o[32];
        dev::tmem_ld32(t_o + cc * 32, o);
        dev::tmem_wait_ld_regs(o);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (real)
            dst[(cc * 8 + i) * rows] =
                make_uint4(__float_as_uint(__uint_as_float(o[4 * i]) * inv_l),
                           __float_as_uint(__uint_as_float(o[4 * i + 1]) * inv_l),
                           __float_as_uint(__uint_as_float(o[4 * i + 2]) * inv_l),
                           __float_as_uint(__uint_as_float(o[4 * i + 3]) * inv_l));
      }
      if (real) {
        const float m_use = m_ref == neg_inf() ? 0.f : m_ref;
        p.ws_lse[out + row] = l == 0.f ? neg_inf() : (m_use + log2f(l)) * 0.69314718055994531f;
      }
    }
    dev::tc_fence_before();
    __syncwarp();
    if (lane == 0) dev::mbar_arrive(dev::smem_u32(&sm.bar_unit_empty[slot]));
  }
}

// ------------------------------------------------------------------------------------------
// thin CTAs
// ------------------------------------------------------------------------------------------
// Tiles pass through one ring in the order in which the tensor core takes them: the keys of a chunk,
// then the values of the chunk before it, so a chunk's softmax has the time of a chunk's products.
__device__ __forceinline__ void thin_produce(const CUtensorMap& tm_q_thin, const CUtensorMap& tm_q_own,
                                             const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                             const Params& p, const Cta& ct) {
  Smem& sm = *ct.sm;
  const int lane = threadIdx.x & 31;
  volatile int* abort = &sm.abort;
  const Pieces pc(p);
  int published = 0, issued = 0;
  bool ok = true;

  struct Source {  // where a chunk's keys are
    const int* table;
    int pages, key0, len, nt, hk;
    uint64_t policy;
  };
  auto stream = [&](const Source& c, bool keys, const CUtensorMap* map_q, int b0, int cols) {
    int page = pc.page(p, c.table, c.pages, c.key0, c.len);
    for (int t = 0; t < c.nt; ++t) {
      const int key0 = c.key0 + t * kTile, cur = page;
      page = t + 1 < c.nt ? pc.page(p, c.table, c.pages, key0 + kTile, c.len) : -2;
      const int s = issued % kThinStages, ph = (issued / kThinStages) ^ 1;
      const int row = pc.row(p, cur, key0);
      if (!(ok = warp_wait(&sm.bar_empty[s], ph, abort))) return;
      const uint32_t bar = dev::smem_u32(&sm.bar_full[s]);
      if (lane == 0) {
        dev::mbar_arrive_expect_tx(bar, pc.bytes(key0, c.len) + (keys ? cols * 256u : 0u));
        if (keys)
          for (int half = 0; half < 2; ++half)
            dev::tma_load_3d(dev::smem_u32(sm.t.q[s]) + half * kQHalfBytes, map_q, bar, half * 64, c.hk * p.G, b0);
      }
      __syncwarp();
      pc.load(keys ? &tm_k : &tm_v, dev::smem_u32(sm.t.tile[s]), bar, cur, row, c.hk, c.policy);
      ++issued;
    }
  };
  Source before;
  before.nt = 0;
  // a run of steps [k0, k1) of one job, as chunks; box: rows of the query box, cols: real ones
  auto run = [&](const int* table, int pages, int len, int hk, int b0, int k0, int k1, const CUtensorMap* map_q,
                 int box, int cols, long long out, uint64_t policy) {
    const int chunks = (k1 - k0 + kChunk - 1) / kChunk;
    for (int i = 0; i < chunks; ++i) {
      const int slot = published % kChunkSlots;
      if (published >= kChunkSlots &&
          !(ok = warp_wait(&sm.bar_chunk_empty[slot], published / kChunkSlots - 1, abort)))
        return;
      Source c;
      c.table = table, c.pages = pages, c.len = len, c.hk = hk, c.policy = policy;
      c.key0 = (k0 + i * kChunk) * kTile;
      c.nt = min(kChunk, k1 - k0 - i * kChunk);
      if (lane == 0) {
        Chunk& d = sm.chunk[slot];
        d.valid = 1;
        d.nt = c.nt;
        d.keys = min(c.nt * kTile, len - c.key0);
        d.cols = cols;
        d.first = i < 2 ? 1 : 0;
        d.last = i + 2 >= chunks ? 1 : 0;
        d.only = chunks == 1 ? 1 : 0;
        d.out = out + (i & 1) * cols;
        __threadfence_block();
        dev::mbar_arrive(dev::smem_u32(&sm.bar_chunk_full[slot]));
      }
      __syncwarp();
      ++published;
      stream(c, true, map_q, b0, box);
      if (!ok) return;
      if (before.nt > 0) stream(before, false, nullptr, 0, 0);
      if (!ok) return;
      before = c;
    }
  };

  int kind = sm.start[0], idx = sm.start[1], c = sm.start[2];
  if (kind == 1) {  // blocks of few sequences against their prefix
    const int thin_seqs = kThinRows / p.G;
    for (; ok && c < ct.hi && idx < p.num_groups; ++idx) {
      const Group g = load_group(p, idx);
      if (g.tiles == 0 || g.rest == 0 || !rest_thin(p, g)) continue;
      const int cost = thin_job(p, g.tiles), b0 = g.b0 + g.full * 2 * p.S;
      for (int hk = 0; ok && c < ct.hi && hk < p.Hkv; ++hk, c += cost) {
        const int k0 = step_at(ct.lo, c, p.thin_cost), k1 = min(g.tiles, step_at(ct.hi, c, p.thin_cost));
        if (k0 >= k1) continue;
        run(p.prefix_table + static_cast<size_t>(idx) * p.max_prefix_pages, p.max_prefix_pages, g.len, hk, b0, k0,
            k1, &tm_q_thin, thin_seqs * p.G, g.rest * p.G,
            p.thin_row0 + 2ll * p.G * p.Hkv * b0 + 2ll * p.G * g.rest * hk +
                static_cast<long long>(ct.index) * kThinCtaRows, prefix_policy());
      }
    }
    if (ok && c < ct.hi) {
      kind = 2;
      idx = 0;
    }
  }
  if (kind == 2) {  // sequences against their own keys
    for (; ok && c < ct.hi && idx < p.B; ++idx) {
      const int len = seq_len(p, idx), tiles = tiles_of(len);
      const int cost = thin_job(p, tiles);
      for (int hk = 0; ok && tiles > 0 && c < ct.hi && hk < p.Hkv; ++hk, c += cost) {
        const int k0 = step_at(ct.lo, c, p.thin_cost), k1 = min(tiles, step_at(ct.hi, c, p.thin_cost));
        if (k0 >= k1) continue;
        run(p.block_table + static_cast<size_t>(idx) * p.max_pages, p.max_pages, len, hk, idx, k0, k1, &tm_q_own,
            p.G, p.G, p.own_row0 + 2ll * p.G * (static_cast<long long>(idx) * p.Hkv + hk + ct.index), own_policy());
      }
    }
  }
  if (ok && before.nt > 0) stream(before, false, nullptr, 0, 0);
  // the end: a chunk that is not valid for each softmax group
  for (int i = 0; ok && i < 2; ++i) {
    const int slot = published % kChunkSlots;
    if (published >= kChunkSlots) ok = warp_wait(&sm.bar_chunk_empty[slot], published / kChunkSlots - 1, abort);
    if (lane == 0 && ok) {
      sm.chunk[slot].valid = 0;
      __threadfence_block();
      dev::mbar_arrive(dev::smem_u32(&sm.bar_chunk_full[slot]));
    }
    ++published;
  }
  __syncwarp();
  if (lane == 0) {
    // ---- drain: the last load into each stage has landed ----
    for (int i = max(0, issued - kThinStages); i < issued; ++i)
      wait_drain(dev::smem_u32(&sm.bar_full[i % kThinStages]), (i / kThinStages) & 1);
  }
}

__device__ __forceinline__ void thin_mma(const Cta& ct) {
  Smem& sm = *ct.sm;
  const int lane = threadIdx.x & 31;
  volatile int* abort = &sm.abort;
  constexpr uint32_t idesc_s = dev::idesc_bf16_f32(kTile, kThinRows, 0, 0);  // K tile, Q: K-major
  constexpr uint32_t idesc_o = dev::idesc_bf16_f32(kD, kThinRows, 1, 0);     // V^T MN-major, P^T K-major
  bool ok = true;
  int used = 0;              // tiles taken from the ring
  int v_nt = 0, v_keys = 0;  // of the chunk whose P V is next
#pragma unroll 1
  for (int c = 0;; ++c) {    // chunk c, then P V of the chunk before
    const int slot = c % kChunkSlots, g = c & 1;
    if (!(ok = warp_wait(&sm.bar_chunk_full[slot], c / kChunkSlots, abort))) break;
    const int valid = sm.chunk[slot].valid, nt = valid ? sm.chunk[slot].nt : 0, keys = sm.chunk[slot].keys;
    __syncwarp();
    if (valid && lane == 0) dev::mbar_arrive(dev::smem_u32(&sm.bar_chunk_empty[slot]));
    // S of this chunk: its columns of tensor memory were read before the P V of the chunk before last
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
      const int s = used % kThinStages;
      if (!(ok = warp_wait(&sm.bar_full[s], used / kThinStages, abort))) break;
      dev::tc_fence_after();
      if (lane == 0) {
        const uint64_t a0 = dev::smem_desc(dev::smem_u32(sm.t.tile[s]), 16, kGroupBytes, dev::kSwizzle128B);
        const uint64_t b0 = dev::smem_desc(dev::smem_u32(sm.t.q[s]), 16, 1024, dev::kSwizzle128B);
#pragma unroll
        for (int ks = 0; ks < kD / 16; ++ks)
          dev::umma_ss(ct.tmem + (g * kChunk + t) * kThinRows, a0 + (((ks >> 2) * kGroupHalf + (ks & 3) * 32) >> 4),
                       b0 + (((ks >> 2) * kQHalfBytes + (ks & 3) * 32) >> 4), idesc_s, ks > 0 ? 1u : 0u);
        dev::umma_commit(dev::smem_u32(&sm.bar_empty[s]));
        if (t == nt - 1) dev::umma_commit(dev::smem_u32(&sm.bar_s[g]));
      }
      __syncwarp();
      ++used;
    }
    if (!ok) break;
    if (c > 0) {
      const int pg = g ^ 1;
      if (!(ok = warp_wait(&sm.bar_p[pg], (c - 1) >> 1, abort))) break;
#pragma unroll 1
      for (int t = 0; t < v_nt; ++t) {
        const int s = used % kThinStages;
        if (!(ok = warp_wait(&sm.bar_full[s], used / kThinStages, abort))) break;
        const uint32_t tile = dev::smem_u32(sm.t.tile[s]);
        const int tail = v_keys - t * kTile;
        if (tail < kTile) zero_tail(tile, tail);
        dev::tc_fence_after();
        if (lane == 0) {
          const uint64_t a0 = dev::smem_desc(tile, kGroupHalf, kGroupBytes, dev::kSwizzle128B);
          const uint64_t b0 = dev::smem_desc(dev::smem_u32(sm.t.p[pg][t]), 16, 1024, dev::kSwizzle128B);
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            dev::umma_ss(ct.tmem + 256 + pg * kThinRows, a0 + ((ks * 2 * kGroupBytes) >> 4),
                         b0 + (((ks >> 2) * kPBlockBytes + (ks & 3) * 32) >> 4), idesc_o, (t > 0 || ks > 0) ? 1u : 0u);
          dev::umma_commit(dev::smem_u32(&sm.bar_empty[s]));
          if (t == v_nt - 1) dev::umma_commit(dev::smem_u32(&sm.bar_o[pg]));
        }
        __syncwarp();
        ++used;
      }
      if (!ok) break;
    }
    if (!valid) break;
    v_nt = nt;
    v_keys = keys;
  }
  __syncwarp();
  if (lane == 0) {
    dev::umma_commit(dev::smem_u32(&sm.bar_drain));
    wait_drain(dev::smem_u32(&sm.bar_drain), 0);
  }
}

// The four warps of a softmax group meet (bounded, like every other wait); n counts the meetings.
__device__ __forceinline__ bool group_sync(Smem& sm, int g, int& n) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) dev::mbar_arrive(dev::smem_u32(&sm.bar_group[g]));
  return warp_wait(&sm.bar_group[g], n++, &sm.abort);
}

// 16 TMEM columns, for tmem_ld_n's other counts see there
template <int N>
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N <= 8) {
    dev::tmem_ld_n<N>(taddr, r);
  } else {
    uint32_t lo[8], hi[8];
    dev::tmem_ld_n<8>(taddr, lo);
    dev::tmem_ld_n<8>(taddr + 8, hi);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = lo[i], r[8 + i] = hi[i];
  }
}

// Reduce N values (a power of two up to 16) over the lanes of a warp, each step exchanging half of the
// values a lane still carries: N + log2(32 / N) - 1 shuffles instead of 5 N.  The lane ends with value
// lane / (32 / N).
template <int N, bool kMax>
__device__ __forceinline__ float reduce_columns(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  auto op = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
  int o = 16;
#pragma unroll
  for (int n = N; n > 1; n >>= 1, o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float give = up ? v[i] : v[n / 2 + i], keep = up ? v[n / 2 + i] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  float x = v[0];
#pragma unroll
  for (; o > 0; o >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// What a softmax group carries through a segment: per column the reference (log2 units), this
// thread's keys' sum, and output column `thread`.
struct ThinState {
  float m[kThinRows], l[kThinRows], o[kThinRows];
  int meetings;
};

// One chunk of N columns (N >= the real ones).  Thread i is key i of every tile, then output column i.
template <int N>
__device__ __forceinline__ bool thin_chunk(const Params& p, const Cta& ct, ThinState& st, const Chunk& d, int g, int c) {
  Smem& sm = *ct.sm;
  const int i = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  volatile int* abort = &sm.abort;
  const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
  const int nt = d.nt, keys = d.keys;
  if (d.first) {
#pragma unroll
    for (int e = 0; e < N; ++e) st.m[e] = neg_inf(), st.l[e] = st.o[e] = 0.f;
  }
  bool ok = warp_wait(&sm.bar_s[g], c >> 1, abort);
  // this thread's key of tile t is one of the chunk's
  auto real = [&](int t) { return t * kTile + i < keys; };
  float mx[N];
#pragma unroll
  for (int e = 0; e < N; ++e) mx[e] = neg_inf();
  if (ok) {
    dev::tc_fence_after();
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
      uint32_t raw[N];
      ld_cols<N>(ct.tmem + lane_off + (g * kChunk + t) * kThinRows, raw);
      dev::tmem_wait_ld_regs(raw);
#pragma unroll
      for (int e = 0; e < N; ++e)
        mx[e] = fmaxf(mx[e], real(t) ? __uint_as_float(raw[e]) * p.c : neg_inf());
    }
  }
  // the chunk's maximum per column: shuffles, then the group's four warps (two buffers in turn)
  float(*red)[kThinRows] = sm.red[g][0][(c >> 1) & 1];
  {
    const float top = reduce_columns<N, true>(mx);
    if (lane % (32 / N) == 0) red[warp][lane / (32 / N)] = top;
  }
  ok = group_sync(sm, g, st.meetings) && ok;
  float alpha[N];
  if (ok) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float top = fmaxf(fmaxf(red[0][e], red[1][e]), fmaxf(red[2][e], red[3][e]));
      const float m = fmaxf(st.m[e], top), use = m == neg_inf() ? 0.f : m;
      alpha[e] = dev::ex2_approx(st.m[e] - use);  // 0 from -inf
      st.m[e] = m;
      st.l[e] *= alpha[e];
      mx[e] = use;
    }
    // P^T[column][key] = 2^(x - m) as bf16: tile t, key block i / 64 (2 KB), row = column (128 bytes),
    // 16-byte chunk (i % 64) / 8 XOR column (the 128-byte swizzle), element i % 8.  Rows of columns
    // that are not real hold anything: they reach only their own columns of O^T.
    const uint32_t kk = static_cast<uint32_t>(i & 63);
    uint8_t* blk = &sm.t.p[g][0][0] + (i >> 6) * kPBlockBytes + (kk & 7) * 2;
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
      uint32_t raw[N];
      ld_cols<N>(ct.tmem + lane_off + (g * kChunk + t) * kThinRows, raw);
      dev::tmem_wait_ld_regs(raw);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float pr = real(t) ? dev::ex2_approx(fmaf(__uint_as_float(raw[e]), p.c, -mx[e])) : 0.f;
        st.l[e] += pr;
        *reinterpret_cast<__nv_bfloat16*>(blk + t * kPTileBytes + e * 128 + ((((kk >> 3) ^ e) & 7) << 4)) =
            __float2bfloat16_rn(pr);
      }
    }
    dev::fence_proxy_async_smem();  // the tensor core reads P through the async proxy
    dev::tc_fence_before();
    __syncwarp();
    if (lane == 0) dev::mbar_arrive(dev::smem_u32(&sm.bar_p[g]));
    ok = warp_wait(&sm.bar_o[g], c >> 1, abort);
  }
  if (ok) {
    dev::tc_fence_after();
    uint32_t o[N];
    ld_cols<N>(ct.tmem + lane_off + 256 + g * kThinRows, o);
    dev::tmem_wait_ld_regs(o);
#pragma unroll
    for (int e = 0; e < N; ++e) st.o[e] = fmaf(st.o[e], alpha[e], __uint_as_float(o[e]));
  }
  if (d.last) {
    // the segment's part: sums over the keys, then O / l and its log-sum-exp
    float(*sums)[kThinRows] = sm.red[g][1][(c >> 1) & 1];
    float l[N];
#pragma unroll
    for (int e = 0; e < N; ++e) l[e] = st.l[e];
    const float sum = reduce_columns<N, false>(l);
    if (lane % (32 / N) == 0) sums[warp][lane / (32 / N)] = sum;
    ok = group_sync(sm, g, st.meetings) && ok;
    if (ok) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float le = sums[0][e] + sums[1][e] + sums[2][e] + sums[3][e];
        if (e < d.cols) p.ws_o[(d.out + e) * kD + i] = le == 0.f ? 0.f : __fdividef(st.o[e], le);
        l[e] = le;
      }
      // thread e writes column e's log-sum-exp, and with a single chunk that of the half that is not there
      if (i < N) {
        float le = 0.f, m = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (i == e) le = l[e], m = st.m[e];
        if (i < d.cols) {
          p.ws_lse[d.out + i] = le == 0.f ? neg_inf() : ((m == neg_inf() ? 0.f : m) + log2f(le)) * 0.69314718055994531f;
          if (d.only) p.ws_lse[d.out + d.cols + i] = neg_inf();
        }
      }
    }
  }
  return ok;
}

__device__ __forceinline__ void thin_softmax(const Params& p, const Cta& ct) {
  Smem& sm = *ct.sm;
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 7;
  volatile int* abort = &sm.abort;
  ThinState st;
  st.meetings = 0;
  bool ok = true;
  for (int c = g; ok; c += 2) {
    const int slot = c % kChunkSlots;
    if (!(ok = warp_wait(&sm.bar_chunk_full[slot], c / kChunkSlots, abort))) break;
    const Chunk& d = sm.chunk[slot];
    if (!d.valid) break;
    switch (d.cols) {
      case 1: ok = thin_chunk<1>(p, ct, st, d, g, c); break;
      case 2: ok = thin_chunk<2>(p, ct, st, d, g, c); break;
      case 3: case 4: ok = thin_chunk<4>(p, ct, st, d, g, c); break;
      case 5: case 6: case 7: case 8: ok = thin_chunk<8>(p, ct, st, d, g, c); break;
      default: ok = thin_chunk<kThinRows>(p, ct, st, d, g, c); break;
    }
    dev::tc_fence_before();
    __syncwarp();
    if (lane == 0) dev::mbar_arrive(dev::smem_u32(&sm.bar_chunk_empty[slot]));
  }
}

// kNeg: the scale is negative, so the largest scaled score comes from the smallest raw score.
template <bool kNeg>
__global__ void __launch_bounds__(kThreads, 1)
    decode_prefix_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_q_thin,
                         const __grid_constant__ CUtensorMap tm_q_own,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- this thread's run of groups and sequences: their cost on the lines ----
  const int per_g = (p.num_groups + kThreads - 1) / kThreads, per_b = (p.B + kThreads - 1) / kThreads;
  const int g0 = min(tid * per_g, p.num_groups), g1 = min(g0 + per_g, p.num_groups);
  const int b0 = min(tid * per_b, p.B), b1 = min(b0 + per_b, p.B);
  int4 mine = make_int4(0, 0, 0, 0);  // wide, thin prefix, own, tiles read from memory
  // (loads of the first group and of the first sequence before either is used)
  const int len0 = b0 < b1 ? seq_len(p, b0) : 0;
  Group first;
  if (g0 < g1) first = load_group(p, g0);
  for (int b = b0; b < b1; ++b) {
    const int tiles = tiles_of(b == b0 ? len0 : seq_len(p, b));
    mine.z += p.Hkv * thin_job(p, tiles);
    mine.w += p.Hkv * tiles;
  }
  bool in_order = true;
  for (int g = g0; g < g1; ++g) {
    in_order = in_order && __ldg(p.group_starts + g) <= __ldg(p.group_starts + g + 1);
    const Group gr = g == g0 ? first : load_group(p, g);
    mine.x += group_wide(p, gr);
    mine.y += group_thin(p, gr);
    mine.w += gr.n > 0 ? p.Hkv * gr.tiles : 0;
  }

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
      dev::mbar_init(dev::smem_u32(&sm.bar_group[s]), 4);
      dev::mbar_init(dev::smem_u32(&sm.bar_unit_full[s]), 1);
      dev::mbar_init(dev::smem_u32(&sm.bar_unit_empty[s]), kUnitReaders);
    }
    for (int s = 0; s < kThinStages; ++s) {
      dev::mbar_init(dev::smem_u32(&sm.bar_full[s]), 1);
      dev::mbar_init(dev::smem_u32(&sm.bar_empty[s]), 1);
    }
    for (int s = 0; s < kChunkSlots; ++s) {
      dev::mbar_init(dev::smem_u32(&sm.bar_chunk_full[s]), 1);
      dev::mbar_init(dev::smem_u32(&sm.bar_chunk_empty[s]), kChunkReaders);
    }
    dev::mbar_init(dev::smem_u32(&sm.bar_drain), 1);
    sm.abort = 0;
    sm.start[0] = 3;  // nothing
    dev::fence_barrier_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    dev::tma_prefetch_desc(&tm_q);
    dev::tma_prefetch_desc(&tm_q_thin);
    dev::tma_prefetch_desc(&tm_q_own);
    dev::tma_prefetch_desc(&tm_k);
    dev::tma_prefetch_desc(&tm_v);
  }
  if (warp == kMmaWarp) {
    dev::tmem_alloc(dev::smem_u32(&sm.tmem_base), 512);
    dev::tmem_relinquish();
  }

  // ---- sums before this thread's run, and of all ----
  int4 run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, run.x, o), y = __shfl_up_sync(0xffffffffu, run.y, o);
    const int z = __shfl_up_sync(0xffffffffu, run.z, o), w = __shfl_up_sync(0xffffffffu, run.w, o);
    if (lane >= o) run.x += x, run.y += y, run.z += z, run.w += w;
  }
  if (lane == 31) sm.scan[warp] = run;
  dev::tc_fence_before();
  // Groups out of order could overlap, and their sums and rows leave their bounds: no prefix counts then.
  const bool ordered = __syncthreads_and(in_order) != 0;
  dev::tc_fence_after();
  int4 all = make_int4(0, 0, 0, 0), at = make_int4(run.x - mine.x, run.y - mine.y, run.z - mine.z, 0);
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int4 s = sm.scan[w];
    if (w < warp) at.x += s.x, at.y += s.y, at.z += s.z;
    all.x += s.x, all.y += s.y, all.z += s.z, all.w += s.w;
  }
  if (!ordered) all.x = all.y = 0;
  at.z += all.y;  // own jobs stand behind the thin prefix jobs
  const int ctas = gridDim.x, cost_wide = all.x, cost_thin = all.y + all.z;
  // The time everything takes, if well divided: what the SMs need, but not less than HBM.  The wide
  // line gets the CTAs that finish it in that time, the thin line the others.
  // Quotients are approximations (an integer division is a hundred clocks of a few on the way to the first
  // load): every CTA computes the same ones, and a share is rounded up past their error.
  const float time = fmaxf(fmaxf(static_cast<float>(all.w) * (static_cast<float>(kHbmNum) / kHbmDen),
                                 __fdividef(static_cast<float>(cost_wide) + static_cast<float>(cost_thin), ctas)),
                           1.f);
  auto split = [](int cost, float by) { return static_cast<int>(__fdividef(static_cast<float>(cost), by) * 1.000001f) + 1; };
  int wide = cost_wide > 0 ? min(split(cost_wide, time), ctas) : 0;
  if (cost_thin > 0) wide = min(wide, ctas - 1);
  if (cost_thin == 0) wide = ctas;
  // every CTA between a job's first and last holds at least one of its steps: a share is not
  // shorter than a step
  const int share_wide = max(wide > 0 ? split(cost_wide, wide) : 0, kCostBoth);
  const int share_thin = max(wide < ctas ? split(cost_thin, ctas - wide) : 0, p.thin_cost);
  // The CTAs of a line stand together: neighbouring SMs share an instruction cache, which holds the code of one
  // kind, not of both.  (In turn over the grid, a wide step took 5400 clocks instead of 4000 and a thin
  // one 3500 instead of 2700, with five times the misses.  For the same reason the loops around the
  // products and over a chunk's tiles are not unrolled: 54 -> 49 us on 97 sequences in 5 groups then.)
  const bool is_wide = static_cast<int>(blockIdx.x) < wide;
  Cta ct;
  ct.sm = &sm;
  ct.tmem = sm.tmem_base;
  ct.index = is_wide ? blockIdx.x : blockIdx.x - wide;
  {
    const int share = is_wide ? share_wide : share_thin, end = is_wide ? cost_wide : cost_thin;
    ct.lo = static_cast<int>(min(static_cast<long long>(ct.index) * share, static_cast<long long>(end)));
    ct.hi = static_cast<int>(min(static_cast<long long>(ct.lo) + share, static_cast<long long>(end)));
  }
  // the job that the share's first position falls into; the first CTA writes the plan down
  const bool writer = blockIdx.x == 0;
  if (writer && tid == 0) {
    p.plan[0] = share_wide;
    p.plan[1] = share_thin;
    p.plan[2] = wide;
    p.plan[3] = ordered ? 1 : 0;
    if (!ordered) atomicExch(&g_device_error, ATTN_ERR_INVALID_ARG);
  }
  auto begins = [&](int kind, int i, int pos, int cost) {
    if (cost > 0 && ct.lo >= pos && ct.lo < pos + cost) {
      sm.start[0] = kind;
      sm.start[1] = i;
      sm.start[2] = pos;
    }
  };
  auto inside = [&](int from, int cost) { return cost > 0 && ct.lo >= from && ct.lo < from + cost; };
  if (ordered && (writer || (is_wide ? inside(at.x, mine.x) : inside(at.y, mine.y)))) {
    int x = at.x, y = at.y;
    for (int g = g0; g < g1; ++g) {
      const Group gr = g == g0 ? first : load_group(p, g);
      const int cx = group_wide(p, gr), cy = group_thin(p, gr);
      if (writer) p.plan[4 + g] = x, p.plan[4 + p.num_groups + g] = y;
      if (is_wide) begins(0, g, x, cx);
      else begins(1, g, y, cy);
      x += cx, y += cy;
    }
  }
  if (writer || (!is_wide && inside(at.z, mine.z))) {
    int z = at.z;
    for (int b = b0; b < b1; ++b) {
      const int cost = p.Hkv * thin_job(p, tiles_of(b == b0 ? len0 : seq_len(p, b)));
      if (writer) p.plan[4 + 2 * p.num_groups + b] = z;
      if (!is_wide) begins(2, b, z, cost);
      z += cost;
    }
  }
  __syncthreads();

  if (warp >= 8) {
    dev::regs_decrease<kRegsOther>();
    if (warp == kLoadWarp) {
      if (is_wide) wide_produce(tm_q, tm_k, tm_v, p, ct);
      else thin_produce(tm_q_thin, tm_q_own, tm_k, tm_v, p, ct);
    } else if (warp == kMmaWarp) {
      if (is_wide) wide_mma(ct);
      else thin_mma(ct);
    }
  } else {
    dev::regs_increase<kRegsSoftmax>();
    if (is_wide) wide_softmax<kNeg>(p, ct);
    else thin_softmax(p, ct);
  }

  // ---- teardown ----
  dev::tc_fence_before();
  __syncthreads();
  // The joining kernel is launched once every CTA is here: earlier, its blocks would all crowd onto
  // the SMs whose CTAs end first.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == kMmaWarp) {
    dev::tc_fence_after();
    dev::tmem_dealloc(ct.tmem, 512);
  }
}

// Join the parts: one block per (kv head, sequence).  A warp takes the G query rows together, so that it
// reads whole sectors of either layout of the parts: lane = row + G * (16-byte column), G warps for all
// columns; kSplit such sets of warps (as many as the SMs hold) share the parts out, 32 / G of them in
// a round.  A round's values are loaded beside its log-sum-exps, not behind them.
// A row's parts from one job are numbered in line order: part e is in the job's e / h-th CTA, h = 2
// where the job's parts come in halves (even and odd steps or chunks; a half that holds nothing has a
// log-sum-exp of -infinity), else 1.
struct Parts {
  int first = 0, ctas = 0, halves = 1;
  int row = 0;           // the part's first row in CTA 0 of the line
  int cta_rows = 0;      // rows from one CTA's part to the next one's
  int half_rows = 0;     // rows from the first half to the second
  int in = 0, rows = 0;  // the first query row within the part; wide: rows of the part, thin: 0
};

// 64 registers, so that an SM holds the 32 warps that the number of sets counts on (97 sequences of 4 kv heads
// 46.7 -> 45.4 us); with fewer query heads that spills, and costs 4% on 23 sequences of one kv head.
template <int G, int kSplit>
__global__ void __launch_bounds__(32 * G * kSplit, G >= 4 ? 32 / (G * kSplit) : 1)
    decode_prefix_combine_kernel(const Params p, __nv_bfloat16* __restrict__ o,
                                 float* __restrict__ lse) {
  constexpr int kRound = 32 / G;                  // parts of a round
  constexpr int kLoads = kRound < 8 ? kRound : 8;  // values on their way at once
  __shared__ float4 sum[kSplit > 1 ? G * kSplit : 1][32];
  __shared__ float2 stat[kSplit > 1 ? kSplit : 1][G];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane % G, part0 = warp / G;
  const int col = (warp % G) * kRound + lane / G;  // in units of 4 columns
  const int hk = blockIdx.x, b = blockIdx.y;

  // ---- inputs of the call: the group of the sequence is the last one that starts at or before it ----
  const int own_tiles = tiles_of(seq_len(p, b));
  int g = -1;
  for (int i0 = 0; i0 < p.num_groups; i0 += 32) {
    const int i = i0 + lane;
    const unsigned m = __ballot_sync(0xffffffffu, i < p.num_groups && __ldg(p.group_starts + i) <= b);
    g += __popc(m);
    if (m != 0xffffffffu) break;
  }
  Group gr;
  if (g >= 0) {
    gr = load_group(p, g);
    if (b >= gr.b0 + gr.n) gr.tiles = 0;
  }
  constexpr int kBlockSeqs = 256 / G;  // 2 S
  const int in = b - (gr.tiles > 0 ? gr.b0 : b), blk = in / kBlockSeqs;
  const bool thin = blk == gr.full && rest_thin(p, gr);
  // ---- what the other kernel left ----
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int share_wide = __ldcg(p.plan), share_thin = __ldcg(p.plan + 1);
  if (__ldcg(p.plan + 3) == 0) gr.tiles = 0;
  const int pos_prefix = gr.tiles > 0 ? __ldcg(p.plan + 4 + (thin ? p.num_groups : 0) + g) : 0;
  const int pos_own = __ldcg(p.plan + 4 + 2 * p.num_groups + b);
  Parts x0, x1;  // of the prefix job, of the own job
  // the CTA that holds position c of a line: a quotient below 149, so one step puts the approximation right
  auto cta_of = [](int c, int share) {
    int q = static_cast<int>(__fdividef(static_cast<float>(c), static_cast<float>(share)));
    if (q * share > c) --q;
    if ((q + 1) * share <= c) ++q;
    return q;
  };
  auto span = [&](Parts& x, int c, int tiles, int w, int share) {
    x.first = cta_of(c, share);
    x.ctas = cta_of(c + (tiles - 1) * w, share) - x.first + 1;
  };
  if (gr.tiles > 0) {
    const int n = blk < gr.full ? kBlockSeqs : gr.rest;
    x0.row = 2 * G * (p.Hkv * (gr.b0 + blk * kBlockSeqs) + n * hk);
    x0.in = (in % kBlockSeqs) * G;
    x0.half_rows = n * G;
    if (thin) {
      x0.halves = 2;
      x0.row += static_cast<int>(p.thin_row0);
      x0.cta_rows = kThinCtaRows;
      x0.rows = 0;
      span(x0, pos_prefix + hk * thin_job(p, gr.tiles), gr.tiles, p.thin_cost, share_thin);
    } else {
      const bool both = n > 128 / G;
      const int w = both ? kCostBoth : kCostAlt;
      x0.halves = both ? 1 : 2;
      x0.cta_rows = kWideCtaRows;
      x0.rows = both ? 128 : n * G;
      if (both && x0.in >= 128) {  // the second row tile's part
        x0.row += 128;
        x0.in -= 128;
        x0.rows = n * G - 128;
      }
      span(x0, pos_prefix + p.Hkv * blk * wide_job(gr.tiles, kCostBoth) + hk * wide_job(gr.tiles, w), gr.tiles, w,
           share_wide);
    }
  }
  if (own_tiles > 0) {
    x1.halves = 2;
    x1.row = static_cast<int>(p.own_row0) + 2 * G * (b * p.Hkv + hk);
    x1.cta_rows = 2 * G;
    x1.half_rows = G;
    x1.rows = x1.in = 0;
    span(x1, pos_own + hk * thin_job(p, own_tiles), own_tiles, p.thin_cost, share_thin);
  }
  const int n0 = x0.halves * x0.ctas, n1 = 2 * x1.ctas;
  const float4* src = reinterpret_cast<const float4*>(p.ws_o);
  float top = neg_inf(), z = 0.f;  // of row r
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int e0 = part0 * kRound; e0 < n0 + n1; e0 += kSplit * kRound) {
    // this lane's part of the round: where its values begin, their step from column to column and from row to
    // row (in units of 4 floats), and row r's log-sum-exp
    int e = e0 + lane / G, at = 0, step = 0, next = 0;
    float L = neg_inf();
    if (e < n0 + n1) {
      const bool first = e < n0;
      if (!first) e -= n0;
      const int halves = first ? x0.halves : 2, h = halves == 2 ? e & 1 : 0, cta = halves == 2 ? e >> 1 : e;
      const int row = (first ? x0.row : x1.row) + ((first ? x0.first : x1.first) + cta) * (first ? x0.cta_rows : x1.cta_rows) +
                      (h ? (first ? x0.half_rows : x1.half_rows) : 0);
      const int rows = first ? x0.rows : 0, inside = first ? x0.in : 0;
      L = __ldcg(p.ws_lse + row + inside + r);
      // a wide part holds 16 bytes of every row after 16 bytes of every row
      at = row * (kD / 4) + (rows > 0 ? inside : inside * (kD / 4));
      step = rows > 0 ? rows : 1;
      next = rows > 0 ? 1 : kD / 4;
    }
    const int parts = min(kRound, n0 + n1 - e0);
#pragma unroll 1
    for (int i0 = 0; i0 < parts; i0 += kLoads) {
      float4 v[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int from = ((i0 + i) * G) & 31;
        const int a = __shfl_sync(0xffffffffu, at, from), st = __shfl_sync(0xffffffffu, step, from);
        const int nx = __shfl_sync(0xffffffffu, next, from);
        v[i] = i0 + i < parts ? src[a + col * st + r * nx] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (i0 == 0) {
        float mx = L;
#pragma unroll
        for (int s = 16; s >= G; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
        const float new_top = fmaxf(top, mx);
        const float f = new_top == neg_inf() ? 1.f : __expf(top - new_top);
        z *= f;
        acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
        top = new_top;
        L = L == neg_inf() ? 0.f : __expf(L - top);  // the part's weight; of NaN parts (NaN inputs) NaN
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const float w = __shfl_sync(0xffffffffu, L, (((i0 + i) * G) & 31) + r);
        if (i0 + i < parts && !(w == 0.f)) {  // a part that holds nothing was never written
          z += w;
          acc.x = fmaf(w, v[i].x, acc.x);
          acc.y = fmaf(w, v[i].y, acc.y);
          acc.z = fmaf(w, v[i].z, acc.z);
          acc.w = fmaf(w, v[i].w, acc.w);
        }
      }
    }
  }
  if constexpr (kSplit > 1) {
    sum[warp][lane] = acc;
    if (warp % G == 0 && lane < G) stat[part0][r] = make_float2(top, z);
    __syncthreads();
    if (part0 != 0) return;
    top = neg_inf();
#pragma unroll
    for (int k = 0; k < kSplit; ++k) top = fmaxf(top, stat[k][r].x);
    z = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kSplit; ++k) {
      const float2 t = stat[k][r];
      const float f = t.x == top ? 1.f : __expf(t.x - top);  // (also where no warp has a part)
      const float4 v = sum[warp + k * G][lane];
      z = fmaf(f, t.y, z);
      acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y), acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
    }
  }
  const long long bh = (static_cast<long long>(b) * p.Hkv + hk) * G + r;
  const float inv = z == 0.f ? 0.f : __fdividef(1.f, z);
  uint2 out;
  out.x = dev::pack_bf16x2(acc.x * inv, acc.y * inv);
  out.y = dev::pack_bf16x2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(o + bh * kD + 4 * col) = out;
  if (col == 0 && lse != nullptr) lse[bh] = z == 0.f ? neg_inf() : top + logf(z);
}

}  // namespace pfx
}  // namespace attn
