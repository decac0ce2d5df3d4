// Attention of one new token a sequence over a paged cache, split over the
// cache's length and joined.
//
// For query head h of sequence b, with x_j = scale log2(e) q.k_j over the rows
// j < lengths[b] on valid pages,
//     o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m),
// in one pass over K and V with the running maximum m. The lengths lie on the
// device, so the split is made there: all tiles (sequence, kv head, 64 keys) in
// one row, an equal share for every CTA, one CTA per SM. A CTA's share is a run
// of pieces, each of one (sequence, kv head); a piece that is not the whole
// head leaves (o, m, sum) in the workspace, and join_kernel puts them together
// in order. Every sum has one order given by the lengths: equal calls give
// equal bits.
//
// Warp 8 feeds a ring of tiles by TMA, one box per run of keys that lies
// together (a page, or what of it divides 64 keys; 128-byte swizzle). Warps 0-3
// and 4-7 take turns at the tiles, 16 keys a warp, and each warp has a softmax
// of its own, so that nothing waits inside a piece; the eight (o, m, sum) are
// joined at its end. Products on the tensor core (mma.sync m16n8k16, fp32
// sums): keys are the rows of S^T = K.Q^T and d the rows of O^T = V^T.P^T, so
// the group's heads fill the 8 columns and one head wastes no more than seven.
// The weights enter P.V as a sum of two numbers of the element type (the first
// rounded towards zero), 16 to 22 bits: the result's own rounding is what is
// left. Bound by HBM: 4 HD bytes a key and kv head, 6 to 16 products each.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "page_ops.h"
#include "ptx.cuh"

namespace lps {
namespace {

constexpr int kTile = 64;          // keys of a tile
constexpr int kConsumers = 8;      // warps of 16 keys; two teams
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kMaxParts = 256;     // CTAs of a launch, and so parts of a head
constexpr int kKid = kKidPagedAttn << 8;

__device__ int g_status[2];        // sticky: error kinds, first report

// fp16 weights are made 2^14 times larger, which the sum divides out, so that
// their second part stays normal.
template <bool BF16>
constexpr float kLift = BF16 ? 0.0f : 14.0f;

template <int HD, int NT>
struct Shape {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kHalf = kTile * 128;             // bytes of 64 keys x 64 elements
  static constexpr int kBytes = kTile * HD * 2;         // K (or V) of a tile
  // Even, so that a stage is always the same team's: a wait for a barrier's phase
  // n by its parity holds only for who knows that phase n - 1 is over, and a team
  // knows that of its own tiles alone.
  static constexpr int kStages = HD == 128 ? 4 : 8;
  static_assert(kStages % 2 == 0, "a stage belongs to one team");
  static constexpr int kRow = HD + 4;                   // floats of a head's row in the join: other banks for other heads
};

template <int HD, int NT>
struct __align__(1024) Smem {
  using S = Shape<HD, NT>;
  uint8_t kv[S::kStages][2][S::kBytes];
  float o[kConsumers][S::kHeads][S::kRow];
  float m[kConsumers][S::kHeads], l[kConsumers][S::kHeads];
  int tiles[kPagedBatch];          // of each sequence
  long long warp_sum[kThreads / 32];
  long long base;                  // first tile of the sequence that the CTA begins in
  int first;                       // that sequence
  int seen[2];                     // whether the piece has a key (pieces take turns)
  uint32_t valid[S::kStages];      // boxes of the tile whose page is one
  uint64_t full[S::kStages], empty[S::kStages];
};

__device__ __forceinline__ void tma_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar,
                                       uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, "
      "%4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar)), "l"(pol)
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
  const int n = __ldcg(p.lengths + b);  // from L2: the join reads it before its wait
  return n > 0 && n <= static_cast<long long>(p.width) * p.page ? n : 0;
}

// The CTAs that have a share, the first tile of CTA c's share of `total` tiles,
// and the CTA that has tile i.
__device__ __forceinline__ int sharers(const PagedAttnParams& p, long long total) {
  return total < p.ctas ? static_cast<int>(total) : p.ctas;
}
__device__ __forceinline__ long long share_start(long long total, int ctas, int c) { return total * c / ctas; }
__device__ __forceinline__ int share_of(long long total, int ctas, long long i) {
  return static_cast<int>(((i + 1) * ctas - 1) / total);
}

// A CTA's pieces in order: tiles [t0, t1) of kv head g of sequence b.
struct Walk {
  long long at, end, base;  // next tile, the share's end, the first tile of sequence b
  int b, nkv;
  const int* tiles;
  int g, t0, t1;
  __device__ __forceinline__ bool next() {
    if (at >= end) return false;
    while (at >= base + static_cast<long long>(nkv) * tiles[b]) {
      base += static_cast<long long>(nkv) * tiles[b];
      ++b;
    }
    const int n = tiles[b];
    const unsigned off = static_cast<unsigned>(at - base);  // below nkv * tiles, kept below 2^31 by the entry point
    g = off / n;
    t0 = off - g * n;
    const long long left = end - at;
    t1 = left < n - t0 ? t0 + static_cast<int>(left) : n;
    at += t1 - t0;
    return true;
  }
};

template <bool BF16, int HD, int NT, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ PagedAttnParams p) {
  using S = Shape<HD, NT>;
  extern __shared__ uint8_t raw[];
  Smem<HD, NT>& sm = *reinterpret_cast<Smem<HD, NT>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kConsumers / 2);
    }
    sm.seen[0] = sm.seen[1] = 0;
    fence_mbar_init();
  }
  // what the stream ran before is done when the join is let start: it may read
  // the lengths at once, and only the parts behind its own wait
  pdl_wait();
  pdl_launch_dependents();

  // the tiles of every sequence, and where this CTA's share begins
  long long total, beg, end;
  {
    const int per = (p.batch + kThreads - 1) / kThreads, lo = min(tid * per, p.batch), hi = min(lo + per, p.batch);
    long long mine = 0;
    for (int b = lo; b < hi; ++b) {
      const int n = (rows_of(p, b) + kTile - 1) / kTile;
      sm.tiles[b] = n;
      mine += n;
    }
    mine *= p.nkv;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    long long before = 0;
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w == warp) before = total;
      total += sm.warp_sum[w];
    }
    const int ctas = sharers(p, total);
    beg = end = total;
    if (static_cast<int>(blockIdx.x) < ctas) beg = share_start(total, ctas, blockIdx.x), end = share_start(total, ctas, blockIdx.x + 1);
    long long at = before + incl - mine;
    if (beg < end && beg >= at && beg < at + mine) {
      int b = lo;
      while (beg >= at + static_cast<long long>(p.nkv) * sm.tiles[b]) at += static_cast<long long>(p.nkv) * sm.tiles[b++];
      sm.first = b;
      sm.base = at;
    }
    __syncthreads();
  }
  if (beg >= end) return;
  Walk walk{beg, end, sm.base, sm.first, p.nkv, sm.tiles, 0, 0, 0};
  const long long limit = wait_cycles(p.wait_limit);

  if (warp == kConsumers) {
    // ---- the ring's producer ----
    const uint64_t pol = l2_evict_first();
    const int boxes = kTile / p.box, box_bytes = p.box * 128, page_boxes = p.page / p.box;
    int it = 0, stage = 0;
    bool ok = true;
    while (ok && walk.next()) {
      const int n_rows = rows_of(p, walk.b);
      const int* table = p.table + static_cast<long long>(walk.b) * p.width;
      const int n_boxes = (n_rows + p.box - 1) / p.box;
      // a lane holds the page of one box; 32 boxes at a time are looked up, one lot ahead
      auto look = [&](int box) {
        if (box >= n_boxes) return make_int2(-1, 0);
        const int pi = box / page_boxes;
        return make_int2(table[pi], (box - pi * page_boxes) * p.box);
      };
      int2 ahead = look(walk.t0 * boxes + lane);
      const int lot = 32 / boxes;  // tiles whose boxes one look covers
      int2 now = ahead;
      for (int t = walk.t0; t < walk.t1; ++t) {
        const int i = (t - walk.t0) % lot;
        if (i == 0) {
          now = ahead;
          ahead = look((t + lot) * boxes + lane);
        }
        if (it >= S::kStages) {
          ok = mbar_wait(&sm.empty[stage], (it / S::kStages - 1) & 1, limit);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        const bool good = now.x >= 0 && now.x < p.n_pages;
        const uint32_t valid = (__ballot_sync(0xffffffffu, good) >> (i * boxes)) & ((1u << boxes) - 1);
        if (lane == 0) {
          sm.valid[stage] = valid;
          mbar_arrive_expect_tx(&sm.full[stage], __popc(valid) * 2 * (HD / 64) * box_bytes);
        }
        __syncwarp();
        // lane: one box of K or V, one half of the head
        constexpr int kParts = 2 * (HD / 64);
        for (int j = lane; __any_sync(0xffffffffu, j < boxes * kParts); j += 32) {
          const int bx = j % boxes, part = j / boxes;
          const int page = __shfl_sync(0xffffffffu, now.x, i * boxes + bx), slot = __shfl_sync(0xffffffffu, now.y, i * boxes + bx);
          if (j < boxes * kParts && (valid >> bx & 1)) {
            const int v = part & 1, half = part >> 1;
            tma_4d(sm.kv[stage][v] + half * S::kHalf + bx * box_bytes, v ? &p.tmap_v : &p.tmap_k, 64 * half, slot, walk.g,
                   page, &sm.full[stage], pol);
          }
        }
        ++it;
        if (++stage == S::kStages) stage = 0;
      }
    }
    if (!ok && lane == 0) report_error(g_status, kErrWaitEmpty | kKid);
    // what is in flight lands before the CTA ends
    for (int i = max(0, it - S::kStages); i < it; ++i)
      if (!mbar_wait(&sm.full[i % S::kStages], (i / S::kStages) & 1, ok ? limit : kDrainLimitCycles)) {
        if (lane == 0) report_error(g_status, kErrDrain | kKid);
        break;
      }
    return;
  }

  // ---- softmax and products: warps 0-7 ----
  const int team = warp >> 2, row0 = (warp & 3) * 16;  // the team's tiles, the warp's keys in a tile
  const int g8 = lane >> 2, t4 = lane & 3;             // fragment coordinates
  const int box_shift = 31 - __clz(p.box);
  bool alive = true;
  int it = 0, piece = 0;
  while (walk.next()) {
    const int n_rows = rows_of(p, walk.b), b = walk.b, g = walk.g;
    // q of the group as the B operand of S^T: column = head
    uint32_t qb[HD / 16][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = 8 * nt + g8;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const char*>(p.q) +
                                                            2 * (b * p.q_seq + static_cast<long long>(g * p.group + h) * p.q_head));
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        qb[kk][nt][0] = h < p.group ? q[8 * kk + t4] : 0u;
        qb[kk][nt][1] = h < p.group ? q[8 * kk + 4 + t4] : 0u;
      }
    }
    float m[NT][2], l[NT][2], o[NT][HD / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int d = 0; d < HD / 16; ++d) o[nt][d][0] = o[nt][d][1] = o[nt][d][2] = o[nt][d][3] = 0.f;
    }
    bool any = false;
    for (int t = walk.t0; t < walk.t1; ++t, ++it) {
      if ((it & 1) != team) continue;
      const int stage = it % S::kStages;
      if (alive) {
        alive = mbar_wait(&sm.full[stage], (it / S::kStages) & 1, limit);
        if (!alive && lane == 0) report_error(g_status, kErrWaitFull | kKid);
        alive = __all_sync(0xffffffffu, alive);
      }
      const int key0 = t * kTile + row0;
      if (alive && key0 < n_rows) {
        // which of the warp's 16 keys there are
        const uint32_t valid = sm.valid[stage];
        const int mine = lane & 15;
        const bool is_key = key0 + mine < n_rows && (valid >> ((row0 + mine) >> box_shift) & 1);
        const uint32_t keys = __ballot_sync(0xffffffffu, is_key) & 0xffffu;
        const uint32_t kbase = smem_u32(sm.kv[stage][0]), vbase = smem_u32(sm.kv[stage][1]);
        const int mtx = lane >> 3, r8 = lane & 7;
        if (keys != 0xffffu) {
          // what lies in the other rows is of no sequence, and 0 x inf is not 0
          for (int c = lane; c < 16 * (HD / 8); c += 32) {
            const int r = c / (HD / 8), ch = c % (HD / 8);
            if (!(keys >> r & 1))
              *reinterpret_cast<uint4*>(sm.kv[stage][1] + (ch / 8) * S::kHalf + (row0 + r) * 128 + (ch % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        }
        if (keys) {
          any = true;
          float s[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
          {
            const int r = row0 + (mtx & 1) * 8 + r8;
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
              uint32_t a[4];
              ldsm_x4(kbase + (kk / 4) * S::kHalf + r * 128 + (((2 * (kk % 4) + (mtx >> 1)) ^ r8) << 4), a);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma<BF16>(s[nt], a, qb[kk][nt][0], qb[kk][nt][1]);
            }
          }
          const bool k0 = keys >> g8 & 1, k1 = keys >> (g8 + 8) & 1;
          uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = (e < 2 ? k0 : k1) ? s[nt][e] * p.scale_log2 : -INFINITY;
            if constexpr (WEIGHTS) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int h = 8 * nt + 2 * t4 + (e & 1), key = key0 + g8 + 8 * (e >> 1);
                if (h < p.group && key < n_rows)
                  p.scores[(static_cast<long long>(b) * p.nq + g * p.group + h) * (static_cast<long long>(p.width) * p.page) + key] = x[e];
              }
            }
            float w[4];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float top = fmaxf(x[c], x[2 + c]);
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
              const float was = m[nt][c], now = fmaxf(was, top);
              const float base = now == -INFINITY ? 0.f : now;
              if (__any_sync(0xffffffffu, now > was)) {  // the whole warp, so that it stays together
                const float f = now > was ? exp2_fast(was - base) : 1.f;
                m[nt][c] = now;
                l[nt][c] *= f;
#pragma unroll
                for (int d = 0; d < HD / 16; ++d) o[nt][d][c] *= f, o[nt][d][2 + c] *= f;
              }
              w[c] = exp2_fast(x[c] - base + kLift<BF16>);
              w[2 + c] = exp2_fast(x[2 + c] - base + kLift<BF16>);
              l[nt][c] += w[c] + w[2 + c];
            }
            uint32_t h0, l0, h1, l1;
            split<BF16>(w[0], w[1], h0, l0);
            split<BF16>(w[2], w[3], h1, l1);
            ph[nt][0] = transposed(h0), ph[nt][1] = transposed(h1);
            pl[nt][0] = transposed(l0), pl[nt][1] = transposed(l1);
          }
          const int r = row0 + (mtx >> 1) * 8 + r8;
#pragma unroll
          for (int d = 0; d < HD / 16; ++d) {
            uint32_t a[4];
            ldsm_x4_t(vbase + (d / 4) * S::kHalf + r * 128 + (((2 * (d % 4) + (mtx & 1)) ^ r8) << 4), a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma<BF16>(o[nt][d], a, ph[nt][0], ph[nt][1]);
              mma<BF16>(o[nt][d], a, pl[nt][0], pl[nt][1]);
            }
          }
        }
        if (keys != 0xffffu) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // zeros before the next copy's bytes
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[stage]);
    }

    // ---- the piece's end: eight warps' (o, m, l) in warp order ----
    named_bar_sync(1, kConsumers * 32);  // the last piece's have been read
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[nt][c];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int h = 8 * nt + 2 * t4 + c;
        if (g8 == 0) sm.m[warp][h] = m[nt][c], sm.l[warp][h] = sum;
#pragma unroll
        for (int d = 0; d < HD / 16; ++d) {
          sm.o[warp][h][16 * d + g8] = o[nt][d][c];
          sm.o[warp][h][16 * d + g8 + 8] = o[nt][d][2 + c];
        }
      }
    if (any && lane == 0) sm.seen[piece & 1] = 1;
    named_bar_sync(1, kConsumers * 32);
    const bool seen = sm.seen[piece & 1] != 0;
    if (tid == 0) sm.seen[~piece & 1] = 0;
    const bool whole = walk.t0 == 0 && walk.t1 == walk.tiles[b];
    const long long slot = (static_cast<long long>(blockIdx.x) * 2 + (piece ? 1 : 0)) * p.group;
    for (int i = tid; i < p.group * HD; i += kConsumers * 32) {
      const int h = i / HD, d = i % HD;
      float top = sm.m[0][h];
#pragma unroll
      for (int w = 1; w < kConsumers; ++w) top = fmaxf(top, sm.m[w][h]);
      const float base = top == -INFINITY ? 0.f : top;
      float sum = 0.f, acc = 0.f;
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) {
        const float f = exp2_fast(sm.m[w][h] - base);
        sum += f * sm.l[w][h];
        acc += f * sm.o[w][h][d];
      }
      const int head = g * p.group + h;
      if (whole) {
        store_out<BF16>(p.out, b * p.o_seq + head * p.o_head + d, seen ? acc / sum : 0.f);
        if (WEIGHTS && d == 0)
          p.part_ml[(2ll * p.ctas + static_cast<long long>(b) * p.nkv + g) * p.group + h] = make_float4(top, sum, 1.f, 0.f);
      } else {
        p.part_o[(slot + h) * HD + d] = acc;
        if (d == 0) p.part_ml[slot + h] = make_float4(top, sum, seen ? 1.f : 0.f, 0.f);
      }
    }
    ++piece;
  }
}

constexpr int kJoin = 256;         // threads of the join
constexpr int kJoinKeys = 1024;    // keys of one of its blocks, with key weights

// Block = (kv head, sequence): the parts of the group's heads that several CTAs
// have computed, in their order; zeros where the sequence has no rows. With key
// weights also the block's share of the cached rows: their weights over the
// group's heads, into the pages' entries.
template <bool BF16, int HD, bool WEIGHTS>
__global__ void __launch_bounds__(kJoin) join_kernel(const __grid_constant__ PagedAttnParams p) {
  __shared__ long long sums[2][kJoin / 32];
  __shared__ float factor[kMaxGroup][kMaxParts];  // 2^(m of the part - m)
  __shared__ float top[kMaxGroup], inv[kMaxGroup];
  __shared__ int seen[kMaxGroup];
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = blockIdx.x, b = blockIdx.y;
  long long before = 0, total = 0;
  for (int i = tid; i < p.batch; i += kJoin) {
    const int n = (rows_of(p, i) + kTile - 1) / kTile;
    total += n;
    if (i < b) before += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (lane == 0) sums[0][warp] = before, sums[1][warp] = total;
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int w = 0; w < kJoin / 32; ++w) before += sums[0][w], total += sums[1][w];
  const int n_rows = rows_of(p, b), n = (n_rows + kTile - 1) / kTile;
  int c0 = 0, c1 = 0;
  bool shifted = false;  // the first part is not its CTA's first piece
  if (n) {
    total *= p.nkv;
    const int ctas = sharers(p, total);
    const long long i0 = before * p.nkv + static_cast<long long>(g) * n;
    c0 = share_of(total, ctas, i0), c1 = share_of(total, ctas, i0 + n - 1);
    shifted = share_start(total, ctas, c0) < i0;
  }
  const int parts = c1 - c0 + 1;
  auto slot = [&](int i, int h) { return (2ll * (c0 + i) + (i == 0 && shifted ? 1 : 0)) * p.group + h; };
  pdl_wait();
  char* out = static_cast<char*>(p.out) + 2 * (b * p.o_seq + static_cast<long long>(g) * p.group * p.o_head);
  if (n == 0) {
    if (blockIdx.z == 0)
      for (int i = tid; i < p.group * HD; i += kJoin) store_out<BF16>(out, i / HD * p.o_head + i % HD, 0.f);
    return;
  }
  if (!WEIGHTS && parts == 1) return;
  if (WEIGHTS && static_cast<long long>(blockIdx.z) * kJoinKeys >= n_rows) return;

  // warp = head: its base, its sum, and what each part is multiplied by
  for (int h = warp; h < p.group; h += kJoin / 32) {
    if (parts == 1) {
      const float4 ml = p.part_ml[(2ll * p.ctas + static_cast<long long>(b) * p.nkv + g) * p.group + h];  // the whole head's
      if (lane == 0) top[h] = ml.x, inv[h] = 1.f / ml.y;
      continue;
    }
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, p.part_ml[slot(i, h)].x);
    m = warp_max(m);
    const float base = m == -INFINITY ? 0.f : m;
    float sum = 0.f, any = 0.f;
    for (int i = lane; i < parts; i += 32) {
      const float4 ml = p.part_ml[slot(i, h)];
      const float f = exp2_fast(ml.x - base);
      factor[h][i] = f;
      sum += f * ml.y;
      any += ml.z;
    }
    sum = warp_sum(sum);
    any = warp_sum(any);
    if (lane == 0) top[h] = m, inv[h] = 1.f / sum, seen[h] = any > 0.f;
  }
  __syncthreads();
  if (parts > 1 && blockIdx.z == 0) {
    for (int i = tid; i < p.group * HD; i += kJoin) {
      const int h = i / HD, d = i % HD;
      float acc = 0.f;
#pragma unroll 8
      for (int c = 0; c < parts; ++c) acc += factor[h][c] * p.part_o[slot(c, h) * HD + d];
      store_out<BF16>(out, h * p.o_head + d, seen[h] ? acc * inv[h] : 0.f);
    }
  }
  if constexpr (WEIGHTS) {
    const long long rows = static_cast<long long>(p.width) * p.page;
    const float* scores = p.scores + (static_cast<long long>(b) * p.nq + g * p.group) * rows;
    // a block's lot of kJoinKeys, and what lies a grid further on
    for (long long lot = static_cast<long long>(blockIdx.z) * kJoinKeys; lot < n_rows; lot += static_cast<long long>(gridDim.z) * kJoinKeys)
    for (int i = tid; i < kJoinKeys && lot + i < n_rows; i += kJoin) {
      const int j = static_cast<int>(lot) + i, pi = j / p.page;
      const int page = p.table[static_cast<long long>(b) * p.width + pi];
      if (page < 0 || page >= p.n_pages) continue;
      float w = 0.f;
      for (int h = 0; h < p.group; ++h) w += exp2_fast(scores[h * rows + j] - top[h] + kLift<BF16>) * inv[h];
      float* to = p.key_weights + (static_cast<long long>(page) * p.nkv + g) * p.page + (j - pi * p.page);
      *to = p.decay == 0.f ? w : p.decay * *to + w;
    }
  }
}

template <class Kern>
cudaError_t launch(Kern kern, dim3 grid, int threads, size_t smem, const PagedAttnParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool BF16, int HD, int NT, bool WEIGHTS>
cudaError_t launch_t(const PagedAttnParams& p, cudaStream_t s) {
  constexpr size_t kSmem = sizeof(Smem<HD, NT>) + 1024;
  static_assert(kSmem <= 232448, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(attn_kernel<BF16, HD, NT, WEIGHTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
  if (e == cudaSuccess) e = launch(attn_kernel<BF16, HD, NT, WEIGHTS>, dim3(p.ctas), kThreads, kSmem, p, s);
  const long long rows = static_cast<long long>(p.width) * p.page;
  const unsigned z = WEIGHTS ? static_cast<unsigned>(rows < 65535ll * kJoinKeys ? (rows + kJoinKeys - 1) / kJoinKeys : 65535) : 1;
  if (e == cudaSuccess) e = launch(join_kernel<BF16, HD, WEIGHTS>, dim3(p.nkv, p.batch, z), kJoin, 0, p, s);
  return e;
}

template <bool BF16, int HD>
cudaError_t launch_g(const PagedAttnParams& p, cudaStream_t s) {
  if (p.group <= 8) return p.key_weights ? launch_t<BF16, HD, 1, true>(p, s) : launch_t<BF16, HD, 1, false>(p, s);
  return p.key_weights ? launch_t<BF16, HD, 2, true>(p, s) : launch_t<BF16, HD, 2, false>(p, s);
}

long long up256(long long x) { return (x + 255) / 256 * 256; }

}  // namespace

cudaError_t paged_attn_ctas(int* ctas) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(ctas, cudaDevAttrMultiProcessorCount, dev);
  if (*ctas > kMaxParts) *ctas = kMaxParts;
  return e;
}

long long paged_attn_workspace(const PagedAttnParams& p, int hd, bool weights) {
  const long long parts = 2ll * p.ctas * p.group;
  long long n = up256(parts * hd * 4) + up256(16 * (parts + (weights ? static_cast<long long>(p.batch) * p.nq : 0)));
  if (weights) n += 4ll * p.batch * p.nq * (static_cast<long long>(p.width) * p.page);
  return n;
}

void paged_attn_place(PagedAttnParams& p, int hd, bool weights, void* workspace) {
  char* at = static_cast<char*>(workspace);
  const long long parts = 2ll * p.ctas * p.group;
  p.part_o = reinterpret_cast<float*>(at);
  at += up256(parts * hd * 4);
  p.part_ml = reinterpret_cast<float4*>(at);
  if (!weights) return;
  at += up256(16 * (parts + static_cast<long long>(p.batch) * p.nq));
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
