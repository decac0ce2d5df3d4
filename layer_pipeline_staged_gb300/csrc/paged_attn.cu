// Attention of one new token a sequence over a paged cache, split over the
// cache's length and joined.
//
// For query head h of sequence b, with x_j = scale log2(e) q.k_j over the rows
// j < lengths[b] on valid pages,
//     o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m),
// in one pass over K and V. m follows the running maximum when that has grown by
// more than 2^8 (o and the sum carry any common factor exactly as well). The
// lengths lie on the device, so the split is made there: the tiles (64 keys) of all
// (sequence, kv head) and a unit for each of these heads, in one row, an equal share
// for every CTA, one CTA per SM. A CTA's share is a run of pieces, each of one head; a
// piece that is not the whole head leaves (o, m, sum) in the workspace, and join_kernel
// puts them together in order. Where the tables have room for few rows of few heads, a
// head is a thread-block cluster's instead: its CTAs take equal runs of the tiles and put
// them together through each other's shared memory, in one launch. Every sum has one order, given by the lengths, the
// batch and the tables' room: equal calls give equal bits (but for the key weights of pages that sequences share, which
// several blocks then write).
//
// Warps 8 and 9 feed a ring of tiles by TMA, one K and one V: a box per run of keys
// that lies together (a page, or what of it divides 64 keys) with both halves of the
// head, 128-byte swizzle; a box takes its warp 50 to 80 cycles to issue, so pages are
// looked up a lot ahead and boxes are as large as pages let them. Warps 0-3 and 4-7
// take turns at the tiles, 16 keys a warp, and each warp has a softmax of its own, so
// that nothing waits inside a piece; warps 10 and 11 join the eight (o, m, sum) at a
// piece's end while the next piece runs. Products on the tensor core (mma.sync
// m16n8k16, fp32 sums; a matrix instruction of 128 rows would have 1 to 16 of them
// used): keys are the rows of S^T = K.Q^T and d the rows of O^T = V^T.P^T, so the
// group's heads fill the 8 columns. The weights enter P.V as a sum of two numbers of
// the element type (the first rounded towards zero), 16 to 22 bits: the result's own
// rounding is what is left.
//
// Bound by HBM: 4 HD bytes a key and kv head against 6 to 16 products each. 24
// sequences of up to 32700 rows, 48/12 heads of 128: 459 us, 6.9 TB/s (the copy rate is
// 6.8); 32 of 0 to 8192, 32/8 heads: 56.5, of which 49.5 are bytes and the rest start, end
// and join; 1000 rows of one: 5.1, latency (7.0 without the cluster). Tried and slower: one producer warp with a
// box per half (the same 32 sequences 110 us), the softmax's warps joining the pieces
// themselves (72), joins by (head, sequence) (72), shares of tiles alone (62), the maximum
// followed in every tile, the join by the last CTA in the same launch (1000 rows 9.5,
// three fences of 900 to 1200 cycles), joins of 512 threads (8.0).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "page_ops.h"
#include "ptx.cuh"

namespace lps {
namespace {

namespace cg = cooperative_groups;

constexpr int kTile = 64;          // keys of a tile
constexpr int kConsumers = 8;      // warps of 16 keys; two teams
constexpr int kProducers = 2;      // warps that feed the ring, one with K and one with V
constexpr int kWriters = 2;        // warps that finish pieces
constexpr int kThreads = (kConsumers + kProducers + kWriters) * 32;
constexpr int kMembers = 8;        // of a cluster at most
constexpr long long kClusterRows = 1024;  // of a member at most
constexpr int kMaxParts = 256;     // CTAs of a launch, and so parts of a head
constexpr int kKid = kKidPagedAttn << 8;
constexpr long long kGiveUp = 1;   // as the wait limit: every wait but those for what is in flight gives up without a look
constexpr float kStale = 8.0f;     // the base may lag the maximum by a factor of 2^8
constexpr uint32_t kWhole = ~0u;   // Smem::valid: all keys of the tile are there

__device__ int g_status[2];        // sticky: error kinds, first report

// fp16 weights are made 2^7 times larger, which the sum divides out: with a stale
// base they reach 2^15, half of the type's range, and their second part stays
// normal further down.
template <bool BF16>
constexpr float kLift = BF16 ? 0.0f : 7.0f;

template <int HD, int NT>
struct Shape {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kBytes = kTile * HD * 2;         // K (or V) of a tile
  // Even, so that a stage is always the same team's: a wait for a barrier's phase
  // n by its parity holds only for who knows that phase n - 1 is over, and a team
  // knows that of its own tiles alone.
  static constexpr int kStages = HD == 128 ? 4 : 8;
  static_assert(kStages % 2 == 0, "a stage belongs to one team");
  static constexpr int kSlots = HD == 128 && NT == 2 ? 1 : 2;  // pieces on their way out
  static constexpr int kQRow = HD * 2 + 16;             // bytes of a head's row of q: other banks for other heads
};

template <int HD, int NT>
struct Slot {
  using S = Shape<HD, NT>;
  float o[kConsumers][NT][HD][8];  // heads side by side, as the fragments hold them
  float m[kConsumers][S::kHeads], l[kConsumers][S::kHeads];
  int seen[kConsumers];            // whether the warp has seen a key
};

template <int HD, int NT>
struct __align__(1024) Smem {
  using S = Shape<HD, NT>;
  uint8_t kv[S::kStages][2][S::kBytes];
  uint8_t q[S::kStages][S::kHeads * S::kQRow];  // of the stages that a team's piece begins with
  Slot<HD, NT> slot[S::kSlots];
  float factor[kWriters][kConsumers][S::kHeads], sum[kWriters][S::kHeads];  // a writer's notes on its piece
  int rows[kPagedBatch];           // of each sequence
  int warp_sum[kThreads / 32];
  int base;                        // first unit of the sequence that the CTA begins in
  int first;                       // that sequence
  uint32_t valid[S::kStages];      // boxes of the tile whose page is one, or kWhole
  float2 part_ml[S::kHeads];       // of a cluster's member: its keys' base and sum (-1: none seen); its o takes the first stage's place
  uint64_t full[S::kStages], empty[S::kStages], slot_full[S::kSlots], slot_empty[S::kSlots];
};

__device__ __forceinline__ void tma_5d(void* dst, const CUtensorMap* map, int y, int z, int w, uint64_t* bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, "
      "%4, %5, %6}], [%7], %8;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(0), "r"(y), "r"(0), "r"(z), "r"(w), "r"(smem_u32(bar)), "l"(pol)
      : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x and y as packed pairs hi + lo of the element type; hi is rounded towards
// zero, so lo keeps the sign of x, and an infinity of V times either is one
// infinity (where lo would be 0, it is the smallest part of x that counts for
// nothing: 0 x inf would be NaN).
template <bool BF16>
__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
  if constexpr (BF16) {
    const uint32_t xb = __float_as_uint(x), yb = __float_as_uint(y);
    hi = __byte_perm(xb, yb, 0x7632);
    const float xl = fmaf(x, 2.3283064e-10f, x - __uint_as_float(xb & 0xffff0000u));  // + x 2^-32
    const float yl = fmaf(y, 2.3283064e-10f, y - __uint_as_float(yb & 0xffff0000u));
    const __nv_bfloat162 v = __floats2bfloat162_rn(xl, yl);
    lo = *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 h = __halves2half2(__float2half_rz(x), __float2half_rz(y));
    hi = *reinterpret_cast<const uint32_t*>(&h);
    const float2 f = __half22float2(h);
    const __half2 v = __floats2half2_rn(fmaf(x, 5.9604645e-8f, x - f.x), fmaf(y, 5.9604645e-8f, y - f.y));  // + x 2^-24
    lo = *reinterpret_cast<const uint32_t*>(&v);
  }
}

template <bool BF16>
__device__ __forceinline__ void store_out(void* out, long long at, float x) {
  if constexpr (BF16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(x);
  else static_cast<__half*>(out)[at] = __float2half_rn(x);
}

// Rows of sequence b: its length, or 0 where that is not one.
__device__ __forceinline__ int rows_of(const PagedAttnParams& p, int b) {
  const int n = __ldcg(p.lengths + b);
  return n > 0 && n <= static_cast<long long>(p.width) * p.page ? n : 0;
}

// What is shared out are units: a head has one for itself (its start and end take
// about as long as a tile) and then one per tile; in 32 bits, the entry point bounds
// them. Without heads' own units, a CTA with a share of one-tile heads took 1.5 times
// as long as the others (32 mixed sequences 62 us).
__device__ __forceinline__ int units_of(int tiles) { return tiles ? tiles + 1 : 0; }

// `total` units in equal shares, the first `more` of one unit more.
struct Shares {
  int ctas, per, more;
  __device__ __forceinline__ Shares(int total, int grid) {
    ctas = max(1, min(total, grid));
    per = total / ctas;
    more = total - per * ctas;
  }
  __device__ __forceinline__ int start(int c) const { return c * per + min(c, more); }
  __device__ __forceinline__ int owner(int unit) const {
    const int head = more * (per + 1);
    return unit < head ? unit / (per + 1) : more + (unit - head) / per;
  }
};

// A CTA's pieces in order: tiles [t0, t1) of kv head g of sequence b.
struct Walk {
  int at, end, base;  // next unit, the share's end, the first unit of sequence b
  int b, nkv;
  const int* rows;
  int g, t0, t1;
  __device__ __forceinline__ int n_rows() const { return rows[b]; }
  __device__ __forceinline__ int tiles() const { return (rows[b] + kTile - 1) / kTile; }
  __device__ __forceinline__ bool next() {
    while (at < end) {
      int n;
      while (n = units_of(tiles()), at >= base + nkv * n) {
        base += nkv * n;
        ++b;
      }
      g = (at - base) / n;
      const int off = at - base - g * n, to = min(n, off + end - at);
      at += to - off;
      t0 = max(off - 1, 0), t1 = to - 1;
      if (t0 < t1) return true;  // else the share ends with the head's own unit
    }
    return false;
  }
};

// The one piece of a cluster's member.
struct OnePiece {
  int rows, b, g, t0, t1;
  bool left;
  __device__ __forceinline__ int n_rows() const { return rows; }
  __device__ __forceinline__ bool next() {
    const bool is = left && t0 < t1;
    left = false;
    return is;
  }
};

// CLUSTER: a (sequence, kv head) is a thread-block cluster's, which shares its tiles out
// and joins them through each other's shared memory: no second launch.
template <bool BF16, int HD, int NT, bool WEIGHTS, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ PagedAttnParams p) {
  using S = Shape<HD, NT>;
  extern __shared__ uint8_t raw[];
  Smem<HD, NT>& sm = *reinterpret_cast<Smem<HD, NT>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sm.full[i], kProducers);
      mbar_init(&sm.empty[i], kConsumers / 2);
    }
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&sm.slot_full[i], kConsumers);
      mbar_init(&sm.slot_empty[i], kWriters);
    }
    fence_mbar_init();
  }
  // heads that the group does not have are columns of zeros
  for (int i = tid; i < static_cast<int>(sizeof sm.q) / 16; i += kThreads) reinterpret_cast<uint4*>(sm.q)[i] = make_uint4(0, 0, 0, 0);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // zeros before the copies' bytes
  if (CLUSTER && tid < S::kHeads) sm.part_ml[tid] = make_float2(-INFINITY, -1.f);
  pdl_wait();
  pdl_launch_dependents();

  // A cluster's member: an equal share of its head's tiles
  OnePiece one{};
  if constexpr (CLUSTER) {
    const int head = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
    one.b = head / p.nkv, one.g = head % p.nkv;
    one.rows = rows_of(p, one.b);
    const int tiles = (one.rows + kTile - 1) / kTile;
    one.t0 = rank * tiles / p.cluster, one.t1 = (rank + 1) * tiles / p.cluster;
    one.left = true;
    __syncthreads();
  }
  // the tiles of every sequence, and where this CTA's share begins
  int beg = 0, end = 0, total = 0;
  if constexpr (!CLUSTER) {
    const int per = (p.batch + kThreads - 1) / kThreads, lo = min(tid * per, p.batch), hi = min(lo + per, p.batch);
    int mine = 0;
    for (int b = lo; b < hi; ++b) {
      const int n = rows_of(p, b);
      sm.rows[b] = n;
      mine += units_of((n + kTile - 1) / kTile);
    }
    mine *= p.nkv;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w == warp) before = total;
      total += sm.warp_sum[w];
    }
    const Shares shares(total, p.ctas);
    beg = end = total;
    if (static_cast<int>(blockIdx.x) < shares.ctas) beg = shares.start(blockIdx.x), end = shares.start(blockIdx.x + 1);
    // the sequence in which the share begins
    int at = before + incl - mine;
    const bool begins = beg < end && beg >= at && beg < at + mine;
    if (begins || (blockIdx.x == 0 && WEIGHTS)) {
      for (int b = lo; b < hi; ++b) {
        const int n = p.nkv * units_of((sm.rows[b] + kTile - 1) / kTile);
        if (WEIGHTS && blockIdx.x == 0) p.first_unit[b] = at;
        if (begins && beg >= at && beg < at + n) sm.first = b, sm.base = at;
        at += n;
      }
    }
    if (beg >= end && tid == 0) p.border[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (WEIGHTS && blockIdx.x == 0 && tid == 0) p.first_unit[p.batch] = total;
    __syncthreads();
  }
  if constexpr (!CLUSTER) {
    // sequences without rows: zeros
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x)
      if (sm.rows[b] == 0)
        for (int i = tid; i < p.nq * HD; i += kThreads) store_out<BF16>(p.out, b * p.o_seq + i / HD * p.o_head + i % HD, 0.f);
    if (beg >= end) return;
  }
  using Pieces = std::conditional_t<CLUSTER, OnePiece, Walk>;
  Pieces walk;
  if constexpr (CLUSTER) walk = one;
  else walk = Walk{beg, end, sm.base, sm.first, p.nkv, sm.rows, 0, 0, 0};
  const long long limit = wait_cycles(p.wait_limit);

  // A warp that gives up a wait says so and ends its role: it arrives nowhere any more,
  // so no barrier's phase is ever completed without what it stands for (no stage is filled
  // again while its copy may be under way, and no writer takes a piece that is not whole),
  // and the waits of the others run out as well.
  auto arrived = [&](uint64_t* bar, int parity, int kind) {
    const bool ok = __all_sync(0xffffffffu, limit != kGiveUp && mbar_wait(bar, parity, limit));
    if (!ok && lane == 0) report_error(g_status, kind | kKid);
    return ok;
  };

  auto roles = [&] {
  if (warp >= kConsumers && warp < kConsumers + kProducers) {
    // ---- the producer of K or of V (and q): what is on its way first takes half the time ----
    const int v = warp - kConsumers;
    const uint64_t pol = l2_evict_first();
    const int log_box = 31 - __clz(p.box), log_boxes = 6 - log_box, boxes = 1 << log_boxes;  // boxes of a tile
    const int page_boxes = p.page >> log_box;
    // a lane's part of a tile: box `lane`
    const int box_bytes = p.box * HD * 2;
    uint8_t* const dst = sm.kv[0][v] + (lane & (boxes - 1)) * box_bytes;
    const CUtensorMap* const map = v ? &p.tmap_v : &p.tmap_k;
    const uint32_t all = (1u << boxes) - 1;
    // Pages of 32 boxes of a sequence, one a lane: (page, row in the page). The
    // next lot of a piece, or the first one of the next piece, is on its way while
    // this one is used.
    const int lot = 32 >> log_boxes;  // tiles of a lot
    auto look = [&](const Pieces& w, int tile) {
      const int box = (tile << log_boxes) + lane;
      if (tile >= w.t1 || box >= (w.n_rows() + p.box - 1) >> log_box) return make_int2(-1, 0);
      const int pi = box / page_boxes;
      return make_int2(p.table[static_cast<long long>(w.b) * p.width + pi], (box - pi * page_boxes) << log_box);
    };
    int it = 0, last = -1;  // tiles of the pieces before; the last one issued
    bool ok = true, more = walk.next();
    int2 ahead = more ? look(walk, walk.t0) : make_int2(-1, 0);
    while (ok && more) {
      Pieces next = walk;
      more = next.next();
      const int n_rows = walk.n_rows(), n_tiles = walk.t1 - walk.t0;
      for (int l0 = 0; l0 < n_tiles && ok; l0 += lot) {
        const int2 now = ahead;
        if (l0 + lot < n_tiles) ahead = look(walk, walk.t0 + l0 + lot);
        else if (more) ahead = look(next, next.t0);
        const uint32_t good = __ballot_sync(0xffffffffu, now.x >= 0 && now.x < p.n_pages);
        const int l1 = min(n_tiles, l0 + lot);
        for (int i = l0; i < l1; ++i) {
          const int stage = (it + i) % S::kStages, use = (it + i) / S::kStages, t = walk.t0 + i;
          if (use) {
            ok = arrived(&sm.empty[stage], (use - 1) & 1, kErrWaitEmpty);
            if (!ok) break;
          }
          const uint32_t valid = good >> ((i - l0) << log_boxes) & all;
          const bool with_q = v == 1 && i < 2;  // a team's first tile of the piece
          const int from = ((i - l0) << log_boxes) + (lane & (boxes - 1));
          const int page = __shfl_sync(0xffffffffu, now.x, from), row = __shfl_sync(0xffffffffu, now.y, from);
          if (lane == 0) {
            if (v == 0) sm.valid[stage] = valid == all && (t + 1) * kTile <= n_rows ? kWhole : valid;
            mbar_arrive_expect_tx(&sm.full[stage], __popc(valid) * box_bytes + (with_q ? p.group * HD * 2 : 0));
          }
          __syncwarp();
          if (with_q && lane < p.group)
            bulk_g2s_plain(sm.q[stage] + lane * S::kQRow,
                           static_cast<const char*>(p.q) + 2 * (walk.b * p.q_seq + static_cast<long long>(walk.g * p.group + lane) * p.q_head),
                           HD * 2, &sm.full[stage]);
          if (lane < boxes && (valid >> lane & 1)) tma_5d(dst + stage * (2 * S::kBytes), map, row, walk.g, page, &sm.full[stage], pol);
          __syncwarp();
          last = it + i;
        }
      }
      it += n_tiles;
      walk = next;
    }
    // What is in flight lands before the CTA ends, whatever limit the waits have and
    // whoever gave up. (A phase that the other producer has not armed does not end; this
    // one's copies have long landed when that wait runs out.)
    bool landed = true;
    for (int i = max(last - (S::kStages - 1), 0); i <= last; ++i)
      landed &= mbar_wait(&sm.full[i % S::kStages], (i / S::kStages) & 1, kDrainLimitCycles);
    if (!__all_sync(0xffffffffu, landed) && lane == 0) report_error(g_status, kErrDrain | kKid);
    return;
  }

  if (warp >= kConsumers + kProducers) {
    // ---- the writers: eight warps' (o, m, l) of a piece, in warp order; warp = half of the elements d ----
    int it = 0;
    const bool tells = warp == kConsumers + kProducers && lane == 0;  // the join of a head that begins here and ends elsewhere
    if (!CLUSTER && tells) p.border[blockIdx.x] = make_int4(0, 0, 0, 0);
    for (int piece = 0; walk.next(); ++piece) {
      const int n = walk.t1 - walk.t0, sl = piece % S::kSlots;
      bool whole = false;
      if constexpr (!CLUSTER) {
        whole = n == walk.tiles();
        if (tells && walk.t0 == 0 && !whole) {
          const int units = walk.tiles() + 1, i0 = walk.base + walk.g * units;
          p.border[blockIdx.x] = make_int4(walk.b, walk.g, Shares(total, p.ctas).owner(i0 + units - 1) - blockIdx.x + 1, beg < i0);
        }
      }
      const int w0 = n == 1 && (it & 1) ? kConsumers / 2 : 0, w1 = n == 1 && !(it & 1) ? kConsumers / 2 : kConsumers;  // the warps that had tiles
      it += n;
      if (!arrived(&sm.slot_full[sl], (piece / S::kSlots) & 1, kErrWaitFull)) return;
      const Slot<HD, NT>& in = sm.slot[sl];
      const long long part = (static_cast<long long>(blockIdx.x) * 2 + (piece ? 1 : 0)) * p.group;
      const int wr = warp - kConsumers - kProducers;
      const bool seen = __any_sync(0xffffffffu, lane >= w0 && lane < w1 && in.seen[lane & 7]);
      // lane = (head, warps w and w + 4): the bases meet, and with them what each warp's part counts
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int h = 8 * nt + (lane & 7), w = lane >> 3;
        const bool on0 = w >= w0 && w < w1, on1 = w + 4 >= w0 && w + 4 < w1;
        const float m0 = on0 ? in.m[w][h] : -INFINITY, m1 = on1 ? in.m[w + 4][h] : -INFINITY;
        float top = fmaxf(m0, m1);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const float base = top == -INFINITY ? 0.f : top;
        const float f0 = exp2_fast(m0 - base), f1 = exp2_fast(m1 - base);
        float sum = (on0 ? f0 * in.l[w][h] : 0.f) + (on1 ? f1 * in.l[w + 4][h] : 0.f);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        sm.factor[wr][w][h] = f0;
        sm.factor[wr][w + 4][h] = f1;
        if (w == 0) {
          sm.sum[wr][h] = sum;
          const float2 ml = make_float2(top, seen ? sum : -1.f);
          if (wr == 0 && h < p.group) {
            if (CLUSTER) sm.part_ml[h] = ml;
            else if (!whole) p.part_ml[part + h] = ml;
            else if (WEIGHTS) p.part_ml[(2ll * p.ctas + static_cast<long long>(walk.b) * p.nkv + walk.g) * p.group + h] = ml;
          }
        }
      }
      __syncwarp();
      // lane = elements d, a writer its half of them, four heads at a time
      constexpr int kEach = HD / kWriters / 32;
#pragma unroll
      for (int h0 = 0; h0 < 8 * NT; h0 += 4) {
        if (h0 >= p.group) break;
        float acc[kEach][4];
#pragma unroll
        for (int e = 0; e < kEach; ++e) acc[e][0] = acc[e][1] = acc[e][2] = acc[e][3] = 0.f;
        for (int w = w0; w < w1; w += kConsumers / 2) {  // a team's warps
#pragma unroll
          for (int j = 0; j < kConsumers / 2; ++j) {
            const float4 f = *reinterpret_cast<const float4*>(&sm.factor[wr][w + j][h0]);
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
              const float4 x = *reinterpret_cast<const float4*>(&in.o[w + j][h0 / 8][(wr * kEach + e) * 32 + lane][h0 % 8]);
              acc[e][0] += f.x * x.x, acc[e][1] += f.y * x.y, acc[e][2] += f.z * x.z, acc[e][3] += f.w * x.w;
            }
          }
        }
        const int d = wr * kEach * 32 + lane;
        if (whole) {
          const long long to = walk.b * p.o_seq + (walk.g * p.group + h0) * p.o_head + d;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (h0 + j >= p.group) break;
            const float inv = seen ? 1.f / sm.sum[wr][h0 + j] : 0.f;  // nothing seen: o is 0
#pragma unroll
            for (int e = 0; e < kEach; ++e) store_out<BF16>(p.out, to + j * p.o_head + 32 * e, acc[e][j] * inv);
          }
        } else {
          float* to = (CLUSTER ? reinterpret_cast<float*>(sm.kv) + h0 * HD : p.part_o + (part + h0) * HD) + d;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (h0 + j >= p.group) break;
#pragma unroll
            for (int e = 0; e < kEach; ++e) to[j * HD + 32 * e] = acc[e][j];
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.slot_empty[sl]);
    }
    return;
  }

  // ---- softmax and products: warps 0-7 ----
  const int team = warp >> 2, row0 = (warp & 3) * 16;  // the team's tiles, the warp's keys in a tile
  const int g8 = lane >> 2, t4 = lane & 3;             // fragment coordinates
  const int mtx = lane >> 3, r8 = lane & 7;            // ldmatrix: matrix and row of the lane's address
  // A box lies as [half of the head][row][128 bytes], its 16-byte units swizzled by the row
  const int box_shift = 31 - __clz(p.box), half = p.box * 128;
  auto place = [&](int row) { return (row >> box_shift) * (p.box * HD * 2) + (row & (p.box - 1)) * 128; };
  const int k_row = place(row0 + (mtx & 1) * 8 + r8), v_row = place(row0 + (mtx >> 1) * 8 + r8);
  int it = 0;
  for (int piece = 0; walk.next(); ++piece) {
    const int b = walk.b, g = walk.g, n_tiles = walk.t1 - walk.t0, sl = piece % S::kSlots;
    float m[NT][2], l[NT][2], o[NT][HD / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int d = 0; d < HD / 16; ++d) o[nt][d][0] = o[nt][d][1] = o[nt][d][2] = o[nt][d][3] = 0.f;
    }
    bool any = false;
    const int skip = (it ^ team) & 1;  // 1: the piece begins with the other team's tile
    uint32_t qb[HD / 16][NT][2];       // q of the group as the B operand of S^T: column = head
    for (int i = skip; i < n_tiles; i += 2) {
      const int t = walk.t0 + i, stage = (it + i) % S::kStages;
      if (!arrived(&sm.full[stage], ((it + i) / S::kStages) & 1, kErrWaitFull)) return;
      if (i < 2) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int kk = 0; kk < HD / 16; kk += 2) {
            uint32_t f[4];
            ldsm_x4(smem_u32(sm.q[stage] + (8 * nt + r8) * S::kQRow + (2 * kk + mtx) * 16), f);
            qb[kk][nt][0] = f[0], qb[kk][nt][1] = f[1], qb[kk + 1][nt][0] = f[2], qb[kk + 1][nt][1] = f[3];
          }
      }
      const int key0 = t * kTile + row0;
      // which of the warp's 16 keys there are
      uint32_t keys = 0xffffu;
      const uint32_t valid = sm.valid[stage];
      if (valid != kWhole) {
        const int mine = lane & 15;
        keys = __ballot_sync(0xffffffffu, key0 + mine < walk.n_rows() && (valid >> ((row0 + mine) >> box_shift) & 1)) & 0xffffu;
      }
      if (keys) {
        any = true;
        const uint32_t kbase = smem_u32(sm.kv[stage][0]) + k_row, vbase = smem_u32(sm.kv[stage][1]) + v_row;
        // S^T in two chains
        float s[NT][4], s2[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < HD / 16; kk += 2) {
          uint32_t a[4], c[4];
          ldsm_x4(kbase + (kk / 4) * half + (((2 * (kk % 4) + (mtx >> 1)) ^ r8) << 4), a);
          ldsm_x4(kbase + (kk / 4) * half + (((2 * (kk % 4) + 2 + (mtx >> 1)) ^ r8) << 4), c);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma<BF16>(s[nt], a, qb[kk][nt][0], qb[kk][nt][1]);
            mma<BF16>(s2[nt], c, qb[kk + 1][nt][0], qb[kk + 1][nt][1]);
          }
        }
        bool above = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = (s[nt][e] + s2[nt][e]) * p.scale_log2;
            s[nt][e] = keys >> (g8 + 8 * (e >> 1)) & 1 ? x : -INFINITY;
            above = above || s[nt][e] > m[nt][e & 1] + kStale;
          }
        if constexpr (WEIGHTS) {
          const long long rows = static_cast<long long>(p.width) * p.page;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int h = 8 * nt + 2 * t4 + (e & 1), key = key0 + g8 + 8 * (e >> 1);
              if (h < p.group && keys >> (g8 + 8 * (e >> 1)) & 1)
                p.scores[(static_cast<long long>(b) * p.nq + g * p.group + h) * rows + key] = s[nt][e];
            }
          __syncwarp();
        }
        // the bases follow the maximum when it has outgrown one of them
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float top = fmaxf(s[nt][c], s[nt][2 + c]);
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
              const float was = m[nt][c], now = fmaxf(was, top);
              const float f = now > was ? exp2_fast(was - now) : 1.f;
              m[nt][c] = now;
              l[nt][c] *= f;
#pragma unroll
              for (int d = 0; d < HD / 16; ++d) o[nt][d][c] *= f, o[nt][d][2 + c] *= f;
            }
        }
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float base = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
            w[e] = exp2_fast(s[nt][e] - base + kLift<BF16>);
            l[nt][e & 1] += w[e];
          }
          uint32_t h0, l0, h1, l1;
          split<BF16>(w[0], w[1], h0, l0);
          split<BF16>(w[2], w[3], h1, l1);
          ph[nt][0] = transposed(h0), ph[nt][1] = transposed(h1);
          pl[nt][0] = transposed(l0), pl[nt][1] = transposed(l1);
        }
        // what lies in the rows that are no keys is of no sequence, and 0 x inf is
        // not 0: where there are such rows, V's fragments lose them
        auto products = [&](auto some) {
          const uint32_t k01 = keys >> (2 * t4), k89 = k01 >> 8;
          const uint32_t lo = (k01 & 1 ? 0xffffu : 0u) | (k01 & 2 ? 0xffff0000u : 0u), hi = (k89 & 1 ? 0xffffu : 0u) | (k89 & 2 ? 0xffff0000u : 0u);
#pragma unroll
          for (int d = 0; d < HD / 16; ++d) {
            uint32_t a[4];
            ldsm_x4_t(vbase + (d / 4) * half + (((2 * (d % 4) + (mtx & 1)) ^ r8) << 4), a);
            if constexpr (decltype(some)::value) a[0] &= lo, a[1] &= lo, a[2] &= hi, a[3] &= hi;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma<BF16>(o[nt][d], a, ph[nt][0], ph[nt][1]);
              mma<BF16>(o[nt][d], a, pl[nt][0], pl[nt][1]);
            }
          }
        };
        if (keys == 0xffffu) products(std::false_type{});
        else products(std::true_type{});
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[stage]);
    }
    it += n_tiles;

    // ---- the piece's end: (o, m, l) to the writers ----
    if (piece >= S::kSlots && !arrived(&sm.slot_empty[sl], (piece / S::kSlots - 1) & 1, kErrWaitEmpty)) return;
    Slot<HD, NT>& out = sm.slot[sl];
    if (skip < n_tiles) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int d = 0; d < HD / 16; ++d) {
          *reinterpret_cast<float2*>(&out.o[warp][nt][16 * d + g8][2 * t4]) = make_float2(o[nt][d][0], o[nt][d][1]);
          *reinterpret_cast<float2*>(&out.o[warp][nt][16 * d + g8 + 8][2 * t4]) = make_float2(o[nt][d][2], o[nt][d][3]);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float sum = l[nt][c];
          sum += __shfl_xor_sync(0xffffffffu, sum, 4);
          sum += __shfl_xor_sync(0xffffffffu, sum, 8);
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          if (g8 == 0) out.m[warp][8 * nt + 2 * t4 + c] = m[nt][c], out.l[warp][8 * nt + 2 * t4 + c] = sum;
        }
      }
      if (lane == 0) out.seen[warp] = any;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.slot_full[sl]);
  }
  };
  roles();

  if constexpr (CLUSTER) {
    // the members' parts in their order, an element of the head's output a thread
    __syncwarp();
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    for (int i = (blockIdx.x % p.cluster) * kThreads + tid; i < p.group * HD; i += p.cluster * kThreads) {
      float2 ml[kMembers];
      float o[kMembers];
#pragma unroll
      for (int r = 0; r < kMembers; ++r) {
        const bool on = r < p.cluster;
        ml[r] = on ? *cluster.map_shared_rank(&sm.part_ml[i / HD], r) : make_float2(-INFINITY, -1.f);
        o[r] = on ? *cluster.map_shared_rank(reinterpret_cast<float*>(sm.kv) + i, r) : 0.f;
      }
      float top = -INFINITY, sum = 0.f, acc = 0.f;
      bool seen = false;
#pragma unroll
      for (int r = 0; r < kMembers; ++r) top = fmaxf(top, ml[r].x);
      const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int r = 0; r < kMembers; ++r) {
        if (ml[r].y < 0.f) continue;  // no key seen, and o is none
        const float w = exp2_fast(ml[r].x - base);
        sum += w * ml[r].y;
        acc += w * o[r];
        seen = true;
      }
      if (WEIGHTS && i % HD == 0)
        p.part_ml[(2ll * p.ctas + static_cast<long long>(one.b) * p.nkv + one.g) * p.group + i / HD] = make_float2(top, seen ? sum : -1.f);
      store_out<BF16>(p.out, one.b * p.o_seq + (one.g * p.group + i / HD) * p.o_head + i % HD, seen ? acc / sum : 0.f);
    }
    cluster.sync();  // a member's parts are read before it ends
  }
}

constexpr int kJoin = 256;         // threads of the join
constexpr int kJoinKeys = 1024;    // keys of one of its blocks that sum key weights
constexpr int kAhead = 8;          // parts that a thread of the join asks for at once

// The place of part i of a head that begins in CTA c0's share, for its query head h.
__device__ __forceinline__ long long part_slot(const PagedAttnParams& p, int c0, bool shifted, int i, int h) {
  return (2ll * (c0 + i) + (i == 0 && shifted ? 1 : 0)) * p.group + h;
}

// Block (CTA c, query head of the group): of the head that begins in CTA c's share
// and ends in another's, the parts in their order. All that a thread reads is asked
// for at once, the parts' bases with their o. With key weights, the other blocks:
// (sequence, kv head, a share of the cached rows), the rows' weights over the
// group's heads into the pages' entries.
template <bool BF16, int HD, bool WEIGHTS>
__global__ void __launch_bounds__(kJoin, 4) join_kernel(const __grid_constant__ PagedAttnParams p, int key_blocks) {
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int joins = p.cluster ? 0 : p.ctas * p.group;
  if (!WEIGHTS || static_cast<int>(blockIdx.x) < joins) {
    constexpr int kSlices = kJoin / HD;  // threads of an element, each with every kSlices-th part
    __shared__ float slice[kSlices][HD], slice_top[kSlices], slice_sum[kSlices], slice_seen[kSlices];
    const int h = blockIdx.x % p.group, d = tid % HD, sl = tid / HD;
    const int c0 = blockIdx.x / p.group;
    pdl_wait();
    const int4 border = __ldcg(p.border + c0);
    const int n = border.z;
    if (n == 0) return;
    float top = -INFINITY, sum = 0.f, acc = 0.f, seen = 0.f;
    for (int i0 = sl; i0 < n; i0 += kAhead * kSlices) {
      float2 ml[kAhead];
      float o[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int part = i0 + i * kSlices;
        const bool on = part < n;
        const long long s = part_slot(p, c0, border.w, on ? part : 0, h);
        ml[i] = on ? __ldcg(p.part_ml + s) : make_float2(-INFINITY, -1.f);
        o[i] = on ? __ldcg(p.part_o + s * HD + d) : 0.f;
      }
      float now = top;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) now = fmaxf(now, ml[i].x);
      const float base = now == -INFINITY ? 0.f : now;
      const float f = exp2_fast(top - base);
      sum *= f, acc *= f, top = now;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (i0 + i * kSlices >= n) break;
        if (ml[i].y < 0.f) continue;  // no key seen
        const float w = exp2_fast(ml[i].x - base);
        sum += w * ml[i].y;
        acc += w * o[i];
        seen = 1.f;
      }
    }
    slice[sl][d] = acc;
    if (d == 0) slice_top[sl] = top, slice_sum[sl] = sum, slice_seen[sl] = seen;
    __syncthreads();
    if (sl) return;
    for (int i = 1; i < kSlices; ++i) top = fmaxf(top, slice_top[i]);
    const float base = top == -INFINITY ? 0.f : top;
    sum = acc = seen = 0.f;
#pragma unroll
    for (int i = 0; i < kSlices; ++i) {
      const float f = exp2_fast(slice_top[i] - base);
      sum += f * slice_sum[i];
      acc += f * slice[i][d];
      seen += slice_seen[i];
    }
    store_out<BF16>(p.out, border.x * p.o_seq + (border.y * p.group + h) * p.o_head + d, seen > 0.f ? acc / sum : 0.f);
    return;
  }
  if constexpr (WEIGHTS) {
    __shared__ float top[kMaxGroup], inv[kMaxGroup];
    const int z = (blockIdx.x - joins) % key_blocks, y = (blockIdx.x - joins) / key_blocks;
    const int b = y / p.nkv, g = y - b * p.nkv;
    const long long first = static_cast<long long>(z) * kJoinKeys;
    pdl_wait();
    const int n_rows = rows_of(p, b);
    if (first >= n_rows) return;
    // the block's keys' pages and scores are asked for before the heads' sums are known
    const long long rows = static_cast<long long>(p.width) * p.page;
    const float* scores = p.scores + (static_cast<long long>(b) * p.nq + g * p.group) * rows;
    const int* table = p.table + static_cast<long long>(b) * p.width;
    constexpr int kKeys = kJoinKeys / kJoin, kEarly = 4;
    float x[kKeys][kEarly];
    int page[kKeys];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const long long key = first + i * kJoin + tid;
      page[i] = key < n_rows ? table[static_cast<int>(key) / p.page] : -1;
#pragma unroll
      for (int h = 0; h < kEarly; ++h) x[i][h] = key < n_rows && h < p.group ? __ldcg(scores + h * rows + key) : 0.f;
    }
    int c0 = 0, n = 1;  // the head's parts: a cluster has put them together
    bool shifted = false;
    if (!p.cluster) {
      const int total = __ldcg(p.first_unit + p.batch), units = units_of((n_rows + kTile - 1) / kTile), i0 = __ldcg(p.first_unit + b) + g * units;
      const Shares shares(total, p.ctas);
      c0 = shares.owner(i0 + 1), n = shares.owner(i0 + units - 1) - c0 + 1;
      shifted = shares.start(c0) < i0;
    }
    for (int h = warp; h < p.group; h += kJoin / 32) {
      float m = -INFINITY, sum = 0.f;
      for (int i = lane; i < n; i += 32) {
        const float2 ml = __ldcg(p.part_ml + (n == 1 ? (2ll * p.ctas + y) * p.group + h : part_slot(p, c0, shifted, i, h)));  // one part: the whole head's
        const float now = fmaxf(m, ml.x), base = now == -INFINITY ? 0.f : now;
        sum = sum * exp2_fast(m - base) + exp2_fast(ml.x - base) * fmaxf(ml.y, 0.f);
        m = now;
      }
      const float all = warp_max(m), base = all == -INFINITY ? 0.f : all;
      sum = warp_sum(sum * exp2_fast(m - base));
      if (lane == 0) top[h] = all, inv[h] = 1.f / sum;
    }
    __syncthreads();
    auto put = [&](long long key, int at, const float (&early)[kEarly]) {
      if (at < 0 || at >= p.n_pages) return;
      float w = 0.f;
#pragma unroll
      for (int h = 0; h < kEarly; ++h)
        if (h < p.group) w += exp2_fast(early[h] - top[h] + kLift<BF16>) * inv[h];
      for (int h = kEarly; h < p.group; ++h) w += exp2_fast(__ldcg(scores + h * rows + key) - top[h] + kLift<BF16>) * inv[h];
      float* to = p.key_weights + (static_cast<long long>(at) * p.nkv + g) * p.page + static_cast<int>(key) % p.page;
      *to = p.decay == 0.f ? w : p.decay * *to + w;
    };
#pragma unroll
    for (int i = 0; i < kKeys; ++i) put(first + i * kJoin + tid, page[i], x[i]);
    // what lies key_blocks further on, where the grid is smaller than the tables
    for (long long lot = first + static_cast<long long>(key_blocks) * kJoinKeys; lot < n_rows; lot += static_cast<long long>(key_blocks) * kJoinKeys)
      for (long long key = lot + tid; key < min(lot + kJoinKeys, static_cast<long long>(n_rows)); key += kJoin) {
        float late[kEarly];
#pragma unroll
        for (int h = 0; h < kEarly; ++h) late[h] = h < p.group ? __ldcg(scores + h * rows + key) : 0.f;
        put(key, table[static_cast<int>(key) / p.page], late);
      }
  }
}

template <bool BF16, int HD, int NT, bool WEIGHTS>
cudaError_t launch_t(const PagedAttnParams& p, cudaStream_t s) {
  constexpr size_t kSmem = sizeof(Smem<HD, NT>) + 1024;
  static_assert(kSmem <= 232448, "shared memory");
  const long long heads = static_cast<long long>(p.batch) * p.nkv, rows = static_cast<long long>(p.width) * p.page;
  // A head is a cluster's where every cluster has a place at once (clusters of eight leave
  // much of the chip unused: 16 of them took 11.1 us for 2000 rows each instead of 7.4 in
  // fours), and the tables have room for so few rows that a member's run costs no more than
  // the second launch. us with clusters and with shares, heads of 128: 1 sequence of 300
  // rows, 8 heads 4.8 and 6.7; of 4000 7.6 and 9.0; of 8000 10.7 and 10.6 (about 1000 rows a
  // member is where they meet), of 16000 17.0 and 13.7; 2 of 4000 10.4 and 10.0; 8 of 2000
  // 10.7 and 13.5; 16 of 500 7.4 and 11.0.
  PagedAttnParams one = p;
  one.cluster = 2 * kMembers * heads <= p.ctas ? kMembers : kMembers / 2;
  while (one.cluster > 1 && one.cluster * heads * 8 > p.ctas * 7) one.cluster /= 2;
  if (one.cluster * heads * 8 > p.ctas * 7 || rows > kClusterRows * one.cluster) one.cluster = 0;
  cudaError_t e;
  if (one.cluster) {
    static std::atomic<uint64_t> told;
    e = allow_smem(attn_kernel<BF16, HD, NT, WEIGHTS, true>, kSmem, told);
    if (e == cudaSuccess)
      e = launch_early_clusters(attn_kernel<BF16, HD, NT, WEIGHTS, true>, dim3(static_cast<unsigned>(one.cluster * heads)), kThreads, kSmem, one.cluster, s, one);
    if (e != cudaSuccess || !WEIGHTS) return e;
  } else {
    static std::atomic<uint64_t> told;
    e = allow_smem(attn_kernel<BF16, HD, NT, WEIGHTS, false>, kSmem, told);
    if (e == cudaSuccess) e = launch_early(attn_kernel<BF16, HD, NT, WEIGHTS, false>, dim3(p.ctas), kThreads, kSmem, s, one);
    if (e != cudaSuccess) return e;
  }
  // blocks for the keys of every head that the tables have room for, in a bounded grid
  const long long lots = (rows + kJoinKeys - 1) / kJoinKeys, most = std::max(1ll, (1ll << 15) / heads);
  const int key_blocks = WEIGHTS ? static_cast<int>(std::min(lots, most)) : 0;
  const long long joins = one.cluster ? 0 : p.ctas * p.group;
  return launch_early(join_kernel<BF16, HD, WEIGHTS>, dim3(static_cast<unsigned>(joins + heads * key_blocks)), kJoin, 0, s, one, key_blocks);
}

template <bool BF16, int HD>
cudaError_t launch_g(const PagedAttnParams& p, cudaStream_t s) {
  if (p.group <= 8) return p.key_weights ? launch_t<BF16, HD, 1, true>(p, s) : launch_t<BF16, HD, 1, false>(p, s);
  return p.key_weights ? launch_t<BF16, HD, 2, true>(p, s) : launch_t<BF16, HD, 2, false>(p, s);
}

long long up256(long long x) { return (x + 255) / 256 * 256; }

}  // namespace

cudaError_t paged_attn_ctas(int* ctas) {
  const cudaError_t e = sm_count(ctas);
  if (*ctas > kMaxParts) *ctas = kMaxParts;
  return e;
}

long long paged_attn_workspace(const PagedAttnParams& p, int hd, bool weights) {
  const long long parts = 2ll * p.ctas * p.group;
  long long n = up256(parts * hd * 4) + up256(8 * (parts + (weights ? static_cast<long long>(p.batch) * p.nq : 0)));
  n += up256(16ll * p.ctas) + up256(4ll * (p.batch + 1));
  if (weights) n += 4ll * p.batch * p.nq * (static_cast<long long>(p.width) * p.page);
  return n;
}

void paged_attn_place(PagedAttnParams& p, int hd, bool weights, void* workspace) {
  char* at = static_cast<char*>(workspace);
  const long long parts = 2ll * p.ctas * p.group;
  p.part_o = reinterpret_cast<float*>(at);
  at += up256(parts * hd * 4);
  p.part_ml = reinterpret_cast<float2*>(at);
  at += up256(8 * (parts + (weights ? static_cast<long long>(p.batch) * p.nq : 0)));
  p.border = reinterpret_cast<int4*>(at);
  at += up256(16ll * p.ctas);
  p.first_unit = reinterpret_cast<int*>(at);
  at += up256(4ll * (p.batch + 1));
  p.scores = reinterpret_cast<float*>(at);
}

cudaError_t launch_paged_attn(const PagedAttnParams& p, bool bf16, int hd, cudaStream_t s) {
  if (hd == 64) return bf16 ? launch_g<true, 64>(p, s) : launch_g<false, 64>(p, s);
  return bf16 ? launch_g<true, 128>(p, s) : launch_g<false, 128>(p, s);
}

cudaError_t paged_attn_status(int* status, cudaStream_t s) {
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  e = cudaMemcpyFromSymbol(status, g_status, 2 * sizeof(int));
  if (e != cudaSuccess || (!status[0] && !status[1])) return e;
  const int zero[2] = {0, 0};
  return cudaMemcpyToSymbol(g_status, zero, sizeof zero);
}

}  // namespace lps
