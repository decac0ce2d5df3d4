// Attention of packed prompts (causal) and of drafted trees over a cache, on
// the fifth-generation tensor cores.
//
// For a query row q and the keys it sees, o = sum_j p_j v_j / sum_j p_j with
// p_j = 2^(x_j - m), x_j = scale log2(e) q.k_j, in one pass over the keys: a
// row keeps the exponent's base m, the sum l of its weights and the unscaled
// o; the base follows the running maximum only when that has grown by more
// than 2^8 (kStale), because o and l carry any common factor exactly as well,
// so o is rescaled a few times per row instead of once per 128 keys.
//
// A tile is 128 rows = the `group` query heads of one kv head x 128 / group
// consecutive tokens, so every key and value fetched serves the whole group,
// and a short sequence still fills the matrix instruction with its heads. A
// CTA runs two such accumulators (slots) at once, so that one slot's softmax
// runs under the other's matrix products:
//   - paired: two neighbouring tiles over the same key blocks (prompts, and
//     trees of more than 128 rows);
//   - solo (trees of up to 128 rows): the one tile over the even and over the
//     odd key blocks; the two halves are joined at the end.
// Per 128-key block and slot: S = Q.K^T (both operands in shared memory,
// 128-byte swizzle, as TMA wrote them) into 128 TMEM columns; four warps read
// a row per thread, make the weights, and write them back over S as the A
// operand of O += P.V, whose B operand is the V block as it lies, keys as rows.
// TMEM: S0 S1 O0 O1.
//
// Warps 0-3 and 4-7: softmax and epilogue of slot 0 and 1. Warp 8: TMA. Warps 9
// and 11: the MMAs of slot 0 and 1. Warp 10: V blocks that some row does not see
// whole are made safe before the MMA reads them, as 0 x inf is not 0: rows past
// the last key become zero, and so do infinities and NaNs, which the epilogue
// then adds to the rows that do see them. Where a row's result is not finite, V is
// looked through again and the formula decides (settle): a weight that came to zero
// in the element type, or a factor that did, leaves NaN of an infinity that counts.
// Finite inputs take neither path.
//
// A prompt's CTA stays on its SM: once the copies of its item are issued, its
// TMA lane takes over the next CTA of the grid that has not started
// (clusterlaunchcontrol), so the next item's Q, K and V arrive, and its first S
// is made, while the last item's softmax and epilogue still run. The grid goes
// through the sequences from the longest to the shortest, and through each from its
// largest item to its smallest.
//
// A tree's keys are shared out over a thread-block cluster, whose CTAs join
// their (o, m, l) through distributed shared memory; a prompt tile's are not.
// Every sum has one order given by the shapes, so equal calls give equal bits.
// Waits are bounded and report through the status word.
//
// What bounds it, on one GB300 (cuBLAS bf16 1865 TFLOP/s, copy 6793 GB/s):
//   - an 8184-token prompt, 32/8 heads of 128: 370 to 374 us, 1470 TFLOP/s. A paired
//     iteration (two tiles x 128 keys) is 2048 cycles of products at the tensor
//     core's rate and takes 2900 to 3300: a block's softmax is 1160 cycles (the
//     hardware's exp2 alone 512), hand-overs between the warps 250 to 300 each,
//     as the products keep shared memory busy (256 KB an iteration at 128 bytes a
//     cycle), and an item's end about 6000 (its last P.V, its rows' way out);
//   - 26 drafts over 8176 rows, 8 kv heads (33.5 MB): 16 us, of which 2.2 until
//     the first S, 6.5 for the blocks, 5 for the join and its barriers.
// Tried and slower: one warp for all MMAs (its waits and commits leave the tensor
// core idle, 428 us), two without turns (they fall into step, 495), P in two halves
// (413), two threads a row (a row's exp2 is bound to its quarter of the SM either
// way, 399), hardware barriers instead of mbarriers (389), output warps of their
// own (too few registers left for the softmax, 410), waits that only spin (385 to
// 399) or that suspend for longer (383), S's upper half ahead (413). Trees of 26
// drafts: one key chunk per CTA with partials in global memory and a merge kernel 22
// us, parts sent to their CTA by stores 16.2, by bulk copies 17.1.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "cache_ops.h"
#include "kernels.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace lps {
namespace {

using namespace tc;

constexpr int kRows = 128;        // rows of a tile (MMA M) and keys of a block (MMA N)
constexpr int kThreads = 384;     // two softmax warpgroups; TMA, two MMA and repair warps
constexpr int kSoftRegs = 208, kOtherRegs = 88;  // 2 * 208 + 88 = 3 * 168, what the block is launched with
constexpr int kLaunchRegs = 168;
constexpr int kMaxStages = 8;
constexpr int kMaxFix = 4;        // blocks of one item that some row does not see whole (at most 3)
constexpr int kClusterSizes = 5;  // clusters of 1, 2, 4, 8 and 16 CTAs
// A prompt launch of up to so many CTAs starts under the stream's last kernel; call
// after call, 32/8 heads of 128: 64 tokens (8 CTAs) 6.1 us so and 6.6 otherwise, 512
// (64) 11.2 and 11.9, 1024 (128) 18.6 and 18.9. With more CTAs than SMs, items of one
// length still gain (2048 tokens, 256 CTAs: 32.3 and 32.7), but of several lengths
// they lose, as early CTAs hold SMs on which the last launch's could take over items
// (7 prompts up to 1024, 296 CTAs: 22.9 and 21.9; 4 up to 1024, 448 CTAs, heads of 64:
// 31.4 and 31.0). A launch of clusters, which take nothing over, always starts so: 1
// row over 1000 8.1 and 9.0, 26 over 8150 15.8 and 16.3, 64 trees of 64 over 4000 237
// and 239.
constexpr int kEarlyCtas = 128;
constexpr float kStale = 8.0f;    // the base may lag the maximum by a factor of about 2^8
// fp16 weights are made 2^7 times larger, which leaves the sum as it is: they reach
// 2^15, half of fp16's range, and stay normal down to 2^-21 of the base and above
// zero down to 2^-32 (2^-14 and 2^-25 without). bf16 has fp32's range.
template <bool BF16>
constexpr float kLift = BF16 ? 0.0f : 7.0f;
constexpr int kKid = kKidTileAttn << 8;

__device__ int g_status[2];       // sticky: error kinds, first report

template <int HD>
struct Shape {
  static constexpr int kTile = kRows * HD * 2;  // bytes of a Q tile, a K block or a V block
  static constexpr int kStages = HD == 128 ? 5 : 8;
  static constexpr int kSmem = (2 + kStages) * kTile + 1024 + (HD == 128 ? 1024 : 1280);  // + alignment + barriers, items and flags
};

// ---- building blocks ---------------------------------------------------------------

__device__ __forceinline__ void tma_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
          "r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// D[tmem] (+)= A[tmem] . B, B in shared memory.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 fp32 columns of this thread's TMEM lane; tmem_wait_ld before they are used.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// 32 columns of 16 TMEM lanes (taddr's on): of lane t / 4 the columns 8i + 2 (t % 4)
// and the next in r[4i] and r[4i + 1], of lane t / 4 + 8 in r[4i + 2] and r[4i + 3].
__device__ __forceinline__ void tmem_ld_quads(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Wait for this thread's loads; v's uses stay behind the wait.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Descriptor of an operand whose rows run along K (V: one key per 128-byte
// row, 64 head dimensions wide): 8-key groups 1024 bytes apart (the stride
// byte offset), the next 64 dimensions one [128 keys][128 bytes] panel on (the
// leading byte offset).
__device__ __forceinline__ uint64_t sw128_desc_rows(uint32_t saddr) {
  uint64_t d = static_cast<uint64_t>((saddr & 0x3ffffu) >> 4);
  d |= static_cast<uint64_t>((kRows * 128) >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// Instruction descriptor as idesc_bf16, for either type, with B's rows along
// K when b_rows (bit 16).
__host__ __device__ constexpr uint32_t idesc_of(bool bf16, int n, bool b_rows) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_rows ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 pack2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(F2 r, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r.v)); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Stores of 32 and 16 bytes by the lanes with `on`, under a predicate: the warp stays together.
__device__ __forceinline__ void st_global32(bool on, void* at, const uint32_t* r) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %9, 0;\n\t"
      "@p st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\t}" ::"l"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(static_cast<uint32_t>(on))
      : "memory");
}
__device__ __forceinline__ void st_global16(bool on, void* at, const uint32_t* r) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %5, 0;\n\t"
      "@p st.global.v4.b32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(static_cast<uint32_t>(on))
      : "memory");
}

// x * 0 + acc: acc becomes NaN where x holds an infinity or a NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t probe(uint32_t x, uint32_t acc) {
  uint32_t r;
  if (BF16)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
  else
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
  return r;
}
template <bool BF16>
__device__ __forceinline__ bool nonfinite(uint32_t half) {  // the low 16 bits
  constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
  return (half & kExp) == kExp;
}
template <bool BF16>
__device__ __forceinline__ float widen(uint16_t x) {
  if (BF16) return __uint_as_float(static_cast<uint32_t>(x) << 16);
  return __half2float(__ushort_as_half(x));
}

// The drafted rows that row t sees, as bits, from parents in [-1, child) or -2
// where that was not so; 0 for a chain that holds a -2.
__device__ __forceinline__ unsigned long long tree_mask(const int8_t* parents, int t) {
  unsigned long long m = 0;
  while (t >= 0) {
    m |= 1ull << t;
    t = parents[t];
  }
  return t == -1 ? m : 0;
}

// Ask for a CTA of this grid that has not started; 16 bytes of answer complete on `bar`.
__device__ __forceinline__ void take_next(void* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
// The index of the CTA taken, or -1 when none is left.
__device__ __forceinline__ int taken(const void* answer) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // read before a later answer is written over it
  return ok ? static_cast<int>(x) : -1;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 peer_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 peer_ld2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- one CTA's work --------------------------------------------------------------

struct Item {
  int idx;           // its CTA in the grid; -1: none is left
  int s, g;          // sequence, kv head
  int len, tok0;     // p.len[s], p.tok0[s]
  int t0;            // first token of slot 0's tile
  int b0, nblk;      // key blocks [b0, b0 + nblk) of this CTA
  int n0, n1;        // of which slots 0 and 1 work through so many (solo: every other one)
  int tiles;         // tiles with rows (1 or 2)
  int clean;         // keys [0, clean) are seen by every row of the item
  int kend;          // keys at and after kend are seen by none
};

template <bool TREE>
__device__ __forceinline__ Item item_of(const TileAttnParams& p, int idx) {
  Item it;
  it.idx = idx;
  const int rank = TREE ? idx % p.cluster : 0, unit = TREE ? idx / p.cluster : idx;
  const int w = unit / p.nkv;
  it.g = unit - w * p.nkv;
  int lo = 0, hi = p.n_seqs - 1;  // the last s with item0[s] <= w
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.item0[mid] <= w) lo = mid; else hi = mid - 1;
  }
  it.s = lo;
  it.len = p.len[lo];
  it.tok0 = p.tok0[lo];
  const int len = it.len, off = w - p.item0[lo], span = 2 * p.tpt;
  if (!TREE) {
    const int pairs = (len + span - 1) / span;
    it.t0 = (pairs - 1 - off) * span;  // the last tokens, which see the most keys, first
    const int endA = min(it.t0 + p.tpt, len), endB = min(it.t0 + span, len);
    it.b0 = 0;
    it.n0 = (endA + kRows - 1) / kRows;
    it.n1 = endB > endA ? (endB + kRows - 1) / kRows : 0;
    it.nblk = max(it.n0, it.n1);
    it.tiles = endB > endA ? 2 : 1;
    it.clean = it.t0 + 1;
    it.kend = endB;
  } else {
    const int all = (p.pos[lo] + len + kRows - 1) / kRows;  // fewer than 2^24, so rank * all fits
    it.t0 = off * span;
    it.b0 = rank * all / p.cluster;
    it.nblk = (rank + 1) * all / p.cluster - it.b0;  // may be none
    it.tiles = it.nblk == 0 ? 0 : !p.solo && it.t0 + p.tpt < len ? 2 : 1;
    it.n0 = p.solo ? (it.nblk + 1) / 2 : it.nblk;
    it.n1 = p.solo ? it.nblk / 2 : it.tiles == 2 ? it.nblk : 0;
    it.clean = p.pos[lo];
    it.kend = p.pos[lo] + len;
  }
  return it;
}

// Which 32 keys from kw on a row sees, as bits. Prompt: the keys [0, lim]; tree:
// the keys [0, lim] and the drafts of anc, whose bit 0 is key lim + 1.
template <bool TREE>
__device__ __forceinline__ uint32_t seen32(int kw, int lim, unsigned long long anc) {
  const int n = lim - kw + 1;
  uint32_t bits = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
  if (TREE) {
    const int d = -n;  // the draft that key kw holds
    if (d >= 0) {
      if (d < 64) bits |= static_cast<uint32_t>(anc >> d);
    } else if (d > -32) {
      bits |= static_cast<uint32_t>(anc << -d);
    }
  }
  return bits;
}

// The weight of a part with (base, sum of weights) ml in a join whose largest
// base is top: 0 where the part saw nothing, NaN where its sum is NaN.
__device__ __forceinline__ float weight_of(float2 ml, float top) {
  if (ml.y == 0.f) return 0.f;
  return ml.y != ml.y ? ml.y : ex2(ml.x - top);
}

// A part of a row with no weight carries a base that says why: the row sees nothing
// by its mask (NaN), the part has had no keys and left no o (-inf), or all its
// scores are -inf and o is 0 times V (0).
__device__ __forceinline__ float2 ml_of_nothing() { return make_float2(NAN, 0.f); }
__device__ __forceinline__ bool sees_nothing(float2 ml) { return ml.y == 0.f && ml.x != ml.x; }
__device__ __forceinline__ float2 ml_without_keys() { return make_float2(-INFINITY, 0.f); }
__device__ __forceinline__ bool has_o(float2 ml) { return ml.y != 0.f || ml.x == 0.f; }

// Whether one of 16-bit words probed into acc is infinite or NaN.
template <bool BF16>
__device__ __forceinline__ bool wild(uint32_t acc) {
  return nonfinite<BF16>(acc) || nonfinite<BF16>(acc >> 16);
}
template <bool BF16>
__device__ __forceinline__ uint32_t probe4(uint4 x, uint32_t acc) {
  return probe<BF16>(x.w, probe<BF16>(x.z, probe<BF16>(x.y, probe<BF16>(x.x, acc))));
}

// The columns of one row's result, 8 (a unit) at a time from unit u0 on, that are not
// finite although the row has weights and no score of it is NaN: where V holds
// infinities or NaNs at keys the row sees, their sum; a key whose score is -inf has a
// weight of zero, and zero times them is NaN; any other weight is positive. Where V
// holds none, the sum has gone past the type, and stays. As no score is NaN or inf, one
// is -inf exactly where the key is not finite. A column is looked for until it is NaN.
template <bool BF16, int HD, bool TREE>
__device__ __forceinline__ void settle(const TileAttnParams& p, const Item& it, int lim, unsigned long long anc, uint16_t* out,
                                       int u0, int step) {
  const uint16_t* k = static_cast<const uint16_t*>(p.k) + it.tok0 * (TREE ? p.k_seq : p.k_row) + it.g * p.k_head;
  const uint16_t* v = static_cast<const uint16_t*>(p.v) + it.tok0 * (TREE ? p.v_seq : p.v_row) + it.g * p.v_head;
#pragma unroll 1
  for (int u = u0; u < HD / 8; u += step) {
    uint32_t open = 0, hit = 0;  // columns that are not finite and not known to be NaN; those of which V says more
#pragma unroll
    for (int e = 0; e < 8; ++e) open |= nonfinite<BF16>(out[u * 8 + e]) ? 1u << e : 0u;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int key = 0; key < it.kend && open; ++key) {
      if (!(seen32<TREE>(key, lim, anc) & 1u)) continue;
      const uint4 x = *reinterpret_cast<const uint4*>(v + key * p.v_row + u * 8);
      if (!wild<BF16>(probe4<BF16>(x, 0))) continue;
      uint32_t acc = 0;
#pragma unroll 1
      for (int d = 0; d < HD; d += 8) acc = probe4<BF16>(*reinterpret_cast<const uint4*>(k + key * p.k_row + d), acc);
      const bool weightless = wild<BF16>(acc);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint16_t y = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
        if (!nonfinite<BF16>(y)) continue;
        sum[e] += weightless ? NAN : widen<BF16>(y);
        hit |= 1u << e;
        if (sum[e] != sum[e]) open &= ~(1u << e);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if ((hit >> e) & 1u) out[u * 8 + e] = static_cast<uint16_t>(pack16<BF16>(sum[e], 0.f));
  }
}

// One row's join over a cluster's C CTAs in order, 8 columns (a unit) at a time
// from unit u0 on: o = sum_c w_c o_c / sum_c w_c l_c, w_c = 2^(m_c - max m). All
// loads of a unit are issued before the first is used: a trip to another CTA's
// shared memory takes some 200 ns, and one per part and unit in turn took 3.5
// of a call's 14 us.
// Returns whether the row's result wants to be settled.
template <bool BF16, int HD, int C>
__device__ __forceinline__ bool join_row(uint32_t ml_at, uint32_t o_at, uint16_t* out, int u0, int step) {
  constexpr int G = C < 8 ? C : 8;  // parts whose loads are under way at once
  float w[C], top = -INFINITY, l = 0.f;
  bool unseen;
  uint32_t has = 0, acc = 0;  // the parts that have left an o; NaN where a result is not finite
  {
    float2 ml[C];
#pragma unroll
    for (int c = 0; c < C; ++c) ml[c] = peer_ld2(peer_smem(ml_at, c));
    unseen = sees_nothing(ml[0]);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (ml[c].y != 0.f) top = fmaxf(top, ml[c].x);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      w[c] = weight_of(ml[c], top);
      has |= has_o(ml[c]) ? 1u << c : 0u;
      if (w[c] != 0.f) l = fmaf(w[c], ml[c].y, l);
    }
  }
  // a draft of a broken chain gets zeros; a row all of whose scores are -inf 0 / 0, as without a join
  const float inv = unseen ? 0.f : l != 0.f ? 1.0f / l : NAN;
  for (int u = u0; u < HD / 8; u += step) {
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < C; g += G) {
      float4 x[G], y[G];
#pragma unroll
      for (int c = 0; c < G; ++c) {
        const uint32_t at = peer_smem(o_at + 2 * u * kRows * 16, g + c);
        x[c] = peer_ld4(at);
        y[c] = peer_ld4(at + kRows * 16);
      }
#pragma unroll
      for (int c = 0; c < G; ++c) {
        const float f = w[g + c];
        if ((has >> (g + c)) & 1u) {  // whatever its weight: zero times an infinity is to be seen
          o[0] = fmaf(f, x[c].x, o[0]);
          o[1] = fmaf(f, x[c].y, o[1]);
          o[2] = fmaf(f, x[c].z, o[2]);
          o[3] = fmaf(f, x[c].w, o[3]);
          o[4] = fmaf(f, y[c].x, o[4]);
          o[5] = fmaf(f, y[c].y, o[5]);
          o[6] = fmaf(f, y[c].z, o[6]);
          o[7] = fmaf(f, y[c].w, o[7]);
        }
      }
    }
    const uint4 y = make_uint4(pack16<BF16>(o[0] * inv, o[1] * inv), pack16<BF16>(o[2] * inv, o[3] * inv),
                               pack16<BF16>(o[4] * inv, o[5] * inv), pack16<BF16>(o[6] * inv, o[7] * inv));
    *reinterpret_cast<uint4*>(out + u * 8) = y;
    acc = probe4<BF16>(y, acc);
  }
  return wild<BF16>(acc) && inv == inv;
}

template <bool BF16, int HD, bool TREE>
__global__ void __launch_bounds__(kThreads, 1) tile_attn_kernel(const __grid_constant__ TileAttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  constexpr int kTile = Shape<HD>::kTile, NS = Shape<HD>::kStages, kPanels = HD / 64, kPanel = kRows * 128;
  static_assert(NS <= kMaxStages, "ring");
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = smem;
  uint8_t* ring = smem + 2 * kTile;
  uint8_t* answer = ring + NS * kTile;                 // [16]: the CTA taken over
  Item* items = reinterpret_cast<Item*>(answer + 16);  // [2]: item number no in place no & 1
  uint64_t* item_full = reinterpret_cast<uint64_t*>(items + 2);  // [2]: the item is there
  uint64_t* item_done = item_full + 2;   // [2]: every role is through with it
  uint64_t* asked = item_done + 2;       // the answer is there
  uint64_t* full = asked + 1;
  uint64_t* empty = full + NS;     // both MMA warps are through with the stage
  uint64_t* qfull = empty + NS;    // [2]: a Q tile is there
  uint64_t* qempty = qfull + 2;    // [2]: its last S is made
  uint64_t* sfull = qempty + 2;    // [2]: S of the slot is ready (and its earlier P.V is done)
  uint64_t* pfull = sfull + 2;     // [2]: P of the slot is written (and O rescaled, and the last item's O read)
  uint64_t* ofull = pfull + 2;     // [2]: the slot's last P.V of the item is done
  uint64_t* vfix = ofull + 2;      // [kMaxFix]: the V block is safe to multiply
  uint64_t* vissued = vfix + kMaxFix;  // [kMaxFix]: its copy has been issued (its stage's phase is the current one)
  uint64_t* mma_done = vissued + kMaxFix;  // [2]
  uint64_t* turn = mma_done + 2;       // [2]: the slot's turn at the tensor core
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(turn + 2);
  volatile int* dirty = reinterpret_cast<int*>(tmem_base + 1);  // [2]: 1 + the last item of that parity with repaired values
  int8_t* parents = reinterpret_cast<int8_t*>(tmem_base + 4);   // [8][kTreeMax], a copy per softmax warp

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool solo = TREE && p.solo;

  pdl_launch_dependents();
  if (tid == 32 * 8) {
    prefetch_map(&p.tmap_q);
    prefetch_map(&p.tmap_k);
    prefetch_map(&p.tmap_v);
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_done[i], 11);  // eight softmax warps, two MMA, repair
      mbar_init(&qfull[i], 1);
      mbar_init(&qempty[i], solo ? 2 : 1);
      mbar_init(&mma_done[i], 1);
      mbar_init(&turn[i], 1);
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 4);
      mbar_init(&ofull[i], 1);
      dirty[i] = 0;
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);
    }
    for (int i = 0; i < kMaxFix; ++i) {
      mbar_init(&vfix[i], 1);
      mbar_init(&vissued[i], 1);
    }
    mbar_init(asked, 1);
    items[0] = item_of<TREE>(p, blockIdx.x);
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_base, 512);
    tmem_relinquish();
  }
  pdl_wait();  // the set-up above runs under the stream's last kernel; all global memory is behind this
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_base;
  const uint32_t tS[2] = {tbase, tbase + 128}, tO[2] = {tbase + 256, tbase + 256 + HD};
  // A tree's result is joined over its cluster (and over the two slots).
  const bool joined = TREE && (solo || p.cluster > 1);
  // After the last product the ring holds what is joined: o [tile][HD / 4][128]
  // float4 columns of rows, the slots' exchange in the second tile's place, and
  // (log2-scaled base, sum of weights) of each slot and of each tile's joined row.
  float4* const join_o = reinterpret_cast<float4*>(ring);
  float4* const swap_o = join_o + HD / 4 * kRows;
  float2* const swap_ml = reinterpret_cast<float2*>(ring + 2 * kRows * HD * 4);
  float2* const join_ml = swap_ml + 2 * kRows;
  static_assert(2 * kRows * HD * 4 + 4 * kRows * 8 <= NS * kTile, "the join fits the ring");

  // first block of an item that some row does not see whole
  auto fix0_of = [](const Item& it) { return max(it.b0, it.clean / kRows); };
  auto blocks_of = [](const Item& it, int slot) { return slot ? it.n1 : it.n0; };
  // Whether there is an item number `no`, which the TMA lane has left in its
  // place (each role for itself would take 1500 cycles to work it out).
  auto item_there = [&](int no) -> bool {
    if (no == 0) return true;
    if (TREE) return false;
    if (!__all_sync(0xffffffffu, mbar_wait(&item_full[no & 1], static_cast<uint32_t>(((no - 1) >> 1) & 1), p.wait_limit))) {
      if (lane == 0) report_error(g_status, kErrWaitFull | kKid | (10 << 13));
      return false;
    }
    return items[no & 1].idx >= 0;
  };
  auto through_with = [&](int no) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_done[no & 1]);
  };

  bool again = false;  // tree: the thread's row wants to be settled
  if (warp >= 8) {
    regs_dec<kOtherRegs>();
    if (warp == 8) {
      // ---------------- TMA ----------------
      if (lane == 0) {
        int n = 0, nq[2] = {0, 0}, nf = 0, asks = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          if (ok && !mbar_wait(bar, parity, p.wait_limit)) {
            report_error(g_status, kErrWaitEmpty | kKid);
            ok = false;
          }
        };
        for (int no = 0; ok; ++no) {
          const Item it = items[no & 1];
          if (it.idx < 0) break;
          const int fix0 = fix0_of(it);
          const int tb = TREE ? 0 : it.tok0, seq = TREE ? it.tok0 : 0;
          auto load = [&](const CUtensorMap* map, int j) {
            const int st = n % NS;
            if (n >= NS) wait(&empty[st], static_cast<uint32_t>((n / NS - 1) & 1));
            if (!ok) return;
            mbar_arrive_expect_tx(&full[st], kTile);
            for (int c = 0; c < kPanels; ++c)
              tma_4d(ring + st * kTile + c * kPanel, map, c * 64, tb + (it.b0 + j) * kRows, it.g, seq, &full[st]);
            ++n;
          };
          for (int t = 0; t < it.tiles; ++t) {
            if (nq[t] > 0) wait(&qempty[t], static_cast<uint32_t>((nq[t] - 1) & 1));
            if (!ok) break;
            ++nq[t];
            mbar_arrive_expect_tx(&qfull[t], static_cast<uint32_t>(p.group * p.tpt) * 128u * kPanels);
            for (int c = 0; c < kPanels; ++c)
              tma_4d(qs + t * kTile + c * kPanel, &p.tmap_q, c * 64, it.g * p.group, tb + it.t0 + t * p.tpt, seq, &qfull[t]);
            if (t == 0) load(&p.tmap_k, 0);
          }
          if (solo && it.nblk > 1) load(&p.tmap_k, 1);
          const int ahead = solo ? 2 : 1;
          for (int j = 0; j < it.nblk && ok; ++j) {
            load(&p.tmap_v, j);
            if (ok && it.b0 + j >= fix0) mbar_arrive(&vissued[nf++ % kMaxFix]);
            if (j + ahead < it.nblk) load(&p.tmap_k, j + ahead);
          }
          if (TREE) break;
          const int place = (no + 1) & 1;  // of the next item; the last but this one was there
          if (ok) {
            mbar_arrive_expect_tx(asked, 16);
            take_next(answer, asked);
            wait(asked, static_cast<uint32_t>(asks++ & 1));
          }
          if (no >= 1) wait(&item_done[place], static_cast<uint32_t>(((no - 1) >> 1) & 1));
          const int idx = ok ? taken(answer) : -1;
          if (idx >= 0) items[place] = item_of<TREE>(p, idx);
          else items[place].idx = -1;
          mbar_arrive(&item_full[place]);
        }
        // every copy issued, and the answer to every take-over asked for, lands
        // before the CTA may end
        bool landed = asks == 0 || mbar_wait(asked, static_cast<uint32_t>((asks - 1) & 1), kDrainLimitCycles);
        for (int t = 0; t < 2; ++t)
          if (nq[t] > 0) landed &= mbar_wait(&qfull[t], static_cast<uint32_t>((nq[t] - 1) & 1), kDrainLimitCycles);
        for (int m = max(n - NS, 0); m < n; ++m)
          landed &= mbar_wait(&full[m % NS], static_cast<uint32_t>((m / NS) & 1), kDrainLimitCycles);
        if (!landed) report_error(g_status, kErrDrain | kKid);
      }
    } else if (warp == 9 || warp == 11) {
      // ---------------- MMA, one warp per slot ----------------
      // Waits and commits cost an issuing thread hundreds of cycles in a row;
      // with a warp per slot they pass under the other slot's products.
      const int slot = warp == 11;
      constexpr uint32_t id_qk = idesc_of(BF16, kRows, false), id_pv = idesc_of(BF16, HD, true);
      bool ok = true;
      int st = 0, nq = 0, np = 0, nf = 0, nt = 0;  // ring stage; Q tiles, P blocks, repaired blocks and turns so far
      uint32_t ph = 0;                     // the stage's phase
      for (int no = 0; item_there(no); ++no) {
        if (lane == 0 && ok) {
          const Item it = items[no & 1];
          const int fix0 = fix0_of(it), mine = blocks_of(it, slot), others = blocks_of(it, slot ^ 1);
          auto wait = [&](uint64_t* bar, uint32_t parity, int what) {
            if (ok && !mbar_wait(bar, parity, p.wait_limit)) {
              report_error(g_status, kErrWaitFull | kKid | (what << 13));
              ok = false;
            }
          };
          auto advance = [&] {
            if (++st == NS) st = 0, ph ^= 1;
          };
          auto wait_p = [&] { wait(&pfull[slot], static_cast<uint32_t>(np++ & 1), 4); };
          auto wait_fix = [&](int j) {
            if (it.b0 + j < fix0) return;
            wait(&vfix[nf % kMaxFix], static_cast<uint32_t>((nf / kMaxFix) & 1), 3);
            ++nf;
          };
          auto skip = [&] {  // a stage that this slot does not use
            wait(&full[st], ph, 1);
            if (ok) mbar_arrive(&empty[st]);
            advance();
          };
          auto qk = [&](int stage, bool both) {
            const uint64_t a = sw128_desc(smem_u32(qs + (solo ? 0 : slot) * kTile)), b = sw128_desc(smem_u32(ring + stage * kTile));
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
              const uint64_t adv = static_cast<uint64_t>((kk / 4) * (kPanel >> 4) + (kk % 4) * 2);
              umma_bf16(tS[slot], a + adv, b + adv, id_qk, kk > 0);
              if (kk == HD / 32 - 1 && both) mbar_arrive(&turn[slot ^ 1]);
            }
            umma_commit(&sfull[slot]);
          };
          auto pv = [&](int stage, bool first) {
            const uint64_t b = sw128_desc_rows(smem_u32(ring + stage * kTile));
#pragma unroll
            for (int kk = 0; kk < kRows / 16; ++kk)  // 16 keys on: 8 columns of P, 2048 bytes of V
              umma_ts(tO[slot], tS[slot] + kk * 8, b + static_cast<uint64_t>(kk * (2048 >> 4)), id_pv, !first || kk > 0);
          };
          // Loads come as K0 V0 K1 V1 .. (paired: every slot takes every block) or
          // K0 K1 V0 K2 V1 K3 .. (solo: slot j & 1 takes block j).
          const int lead = solo ? 2 : 1;
          int done = 0;  // of this slot's blocks, those whose S is under way
          if (it.tiles > (solo ? 0 : slot)) wait(&qfull[solo ? 0 : slot], static_cast<uint32_t>(nq++ & 1), 2);
          for (int j = 0; j < lead && j < it.nblk && ok; ++j) {
            if (solo ? j != slot : mine == 0) {
              skip();
              continue;
            }
            wait(&full[st], ph, 1);
            if (!ok) break;
            tc_fence_after();
            qk(st, false);
            umma_commit(&empty[st]);
            advance();
            if (++done == mine) umma_commit(&qempty[solo ? 0 : slot]);
          }
          if (solo && mine == 0 && ok) mbar_arrive(&qempty[0]);
          for (int j = 0; j < it.nblk && ok; ++j) {
            const bool has_k = j + lead < it.nblk;
            if (solo ? (j & 1) != slot : j >= mine) {
              skip();
              if (it.b0 + j >= fix0) ++nf;
              if (has_k) skip();
              continue;
            }
            const int sv = st;
            wait(&full[st], ph, 1);
            wait_fix(j);
            advance();
            const bool more = done < mine;  // another S of this slot behind this P.V
            const int sk = st;
            if (more) {
              wait(&full[st], ph, 1);
              advance();
            }
            wait_p();
            // The slots take turns at the tensor core, so that they stay half an
            // iteration apart: left to themselves they fall into step, both
            // in their softmax, then both waiting for it. The turn is handed
            // on in the middle of S, to cover the time it takes to arrive.
            // In a paired item they have block j one after the other, in a solo
            // one block j and block j + 1.
            const bool both = solo ? it.nblk > 1 : j < others, give = solo ? j + 1 < it.nblk : both;
            if (both) {
              if (slot == 1 || nt > 0) wait(&turn[slot], static_cast<uint32_t>((slot == 1 ? nt : nt - 1) & 1), 8);
              ++nt;
            }
            if (!ok) break;
            tc_fence_after();
            pv(sv, j < lead);
            if (more) {
              qk(sk, give);
              if (++done == mine) umma_commit(&qempty[solo ? 0 : slot]);
              umma_commit(&empty[sv]);
              umma_commit(&empty[sk]);
            } else {
              if (give) mbar_arrive(&turn[slot ^ 1]);
              umma_commit(&ofull[slot]);
              umma_commit(&empty[sv]);
              if (has_k) skip();
            }
          }
        }
        through_with(no);
      }
      // every MMA has completed before TMEM is freed
      if (lane == 0) {
        umma_commit(&mma_done[slot]);
        if (!mbar_wait(&mma_done[slot], 0, kDrainLimitCycles)) report_error(g_status, kErrDrain | kKid | (1 << 13));
      }
    } else if (warp == 10) {
      // ---------------- V blocks made safe ----------------
      bool ok = true;
      int n0 = 0, nf = 0;
      for (int no = 0; item_there(no); ++no) {
        const Item it = items[no & 1];
        const int fix0 = fix0_of(it);
        for (int kb = fix0; kb < it.b0 + it.nblk && ok; ++kb, ++nf) {
          // place in the load order of V block j of the item: K blocks are ahead of their V
          const int j = kb - it.b0;
          const int n = n0 + (!solo ? 2 * j + 1 : j <= it.nblk - 2 ? 2 * j + 2 : 2 * it.nblk - 1);
          ok = __all_sync(0xffffffffu, mbar_wait(&vissued[nf % kMaxFix], static_cast<uint32_t>((nf / kMaxFix) & 1), p.wait_limit) &&
                                           mbar_wait(&full[n % NS], static_cast<uint32_t>((n / NS) & 1), p.wait_limit));
          if (!ok) {
            if (lane == 0) report_error(g_status, kErrWaitFull | kKid | (5 << 13));
            break;
          }
          uint8_t* v = ring + (n % NS) * kTile;
          const int rows = max(0, min(kRows, it.kend - kb * kRows));  // rows that hold keys
          uint32_t acc[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < kPanels; ++c) {
            uint8_t* panel = v + c * kPanel;
            for (int i = lane + rows * 8; i < kRows * 8; i += 32) reinterpret_cast<uint4*>(panel)[i] = make_uint4(0, 0, 0, 0);
#pragma unroll 8
            for (int i = lane; i < rows * 8; i += 32) {
              const uint4 x = reinterpret_cast<const uint4*>(panel)[i];
              acc[0] = probe<BF16>(x.x, acc[0]);
              acc[1] = probe<BF16>(x.y, acc[1]);
              acc[2] = probe<BF16>(x.z, acc[2]);
              acc[3] = probe<BF16>(x.w, acc[3]);
            }
          }
          bool bad = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) bad |= nonfinite<BF16>(acc[i]) || nonfinite<BF16>(acc[i] >> 16);
          if (__any_sync(0xffffffffu, bad)) {
            for (int c = 0; c < kPanels; ++c)
              for (int i = lane; i < rows * 32; i += 32) {
                uint32_t* w = reinterpret_cast<uint32_t*>(v + c * kPanel) + i;
                uint32_t x = *w;
                if (nonfinite<BF16>(x)) x &= 0xffff0000u;
                if (nonfinite<BF16>(x >> 16)) x &= 0xffffu;
                *w = x;
              }
            if (lane == 0) dirty[no & 1] = no + 1;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the tensor core reads through the async proxy
          __syncwarp();
          if (lane == 0) mbar_arrive(&vfix[nf % kMaxFix]);
        }
        n0 += 2 * it.nblk;
        through_with(no);
      }
    }
  } else {
    // ---------------- softmax and epilogue of slot `slot` ----------------
    regs_inc<kSoftRegs>();
    const int slot = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int row_tok = r / p.group, row_head = r % p.group;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_addr = tS[slot] + lane_off, o_addr = tO[slot] + lane_off;
    const float sl2 = p.scale_log2, slack = kStale / sl2;  // in units of S
    bool ok = true;
    int ns = 0, no_o = 0;  // S blocks and finished accumulators so far
    for (int no = 0; ok && item_there(no); ++no) {
      const Item& it = items[no & 1];
      const int fix0 = fix0_of(it), b0 = it.b0;
      const int len = it.len;
      const int tok = it.t0 + (solo ? 0 : slot * p.tpt) + row_tok;
      const bool row_ok = row_tok < p.tpt && tok < len;
      const bool warp_ok = __any_sync(0xffffffffu, row_ok);
      unsigned long long anc = 0;
      if (TREE) {
        int8_t* mine = parents + warp * kTreeMax;
        __syncwarp();  // the last item's copy has been read
        for (int t = lane; t < len; t += 32) {
          const int up = p.parents[static_cast<size_t>(it.tok0) * p.width + t];
          mine[t] = static_cast<int8_t>(up >= -1 && up < t ? up : -2);
        }
        __syncwarp();
        if (row_ok) anc = tree_mask(mine, tok);
      }
      const int lim = TREE ? p.pos[it.s] - 1 : min(tok, len - 1);
      const int nb = blocks_of(it, slot);
      // the row's base, sum, kLift - base sl2 and the maximum that moves the base,
      // which a row decides for itself: what its warp's other rows see changes nothing
      float m = -INFINITY, l = 0.f, neg = 0.f, bar = -INFINITY;
      auto rebase = [&](float to) {
        m = to;
        neg = to == -INFINITY ? 0.f : fmaf(-to, sl2, kLift<BF16>);
        bar = to + slack;
      };
      for (int i = 0; i < nb && ok; ++i, ++ns) {
        const int kb = b0 + (solo ? 2 * i + slot : i);
        ok = __all_sync(0xffffffffu, mbar_wait(&sfull[slot], static_cast<uint32_t>(ns & 1), p.wait_limit));
        if (!ok) {
          if (lane == 0) report_error(g_status, kErrWaitFull | kKid | (6 << 13));
          break;
        }
        tc_fence_after();
        if (warp_ok) {
          float x[kRows];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, x + c * 32);
          tmem_wait_ld<kRows>(x);
          if (kb >= fix0) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t bits = seen32<TREE>(kb * kRows + c * 32, lim, anc);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((bits >> e) & 1u)) x[c * 32 + e] = -INFINITY;
            }
          }
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int e = 4; e < kRows; e += 8) {
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], x[e + q], e + 4 + q < kRows ? x[e + 4 + q] : x[e + q]);
          }
          const float block = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          if (i == 0) {
            rebase(block);
          } else if (__any_sync(0xffffffffu, row_ok && block > bar)) {  // rows without a query have no say
            // O holds the blocks before this one, whole: S of this block was
            // issued behind their P.V
            const bool stale = block > bar;
            const float f = stale ? ex2((m - block) * sl2) : 1.0f;
            l *= f;
            rebase(stale ? block : m);
            __syncwarp();
#pragma unroll 1
            for (int c = 0; c < HD; c += 32) {
              float o[32];
              tmem_ld32(o_addr + c, o);
              tmem_wait_ld<32>(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= f;
              tmem_st16(o_addr + c, reinterpret_cast<const uint32_t*>(o));
              tmem_st16(o_addr + c + 16, reinterpret_cast<const uint32_t*>(o) + 16);
            }
          }
          const F2 sl = pack2(sl2, sl2), ng = pack2(neg, neg);
          F2 sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float a, b;
              unpack2(fma2(pack2(x[c * 32 + 2 * e], x[c * 32 + 2 * e + 1]), sl, ng), a, b);
              a = ex2(a);
              b = ex2(b);
              sum[e & 1] = add2(sum[e & 1], pack2(a, b));
              w[e] = pack16<BF16>(a, b);
            }
            tmem_st16(s_addr + c * 16, w);
          }
          float a, b;
          unpack2(add2(sum[0], sum[1]), a, b);
          l += a + b;
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[slot]);
      }
      if (nb > 0 && ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ofull[slot], static_cast<uint32_t>(no_o & 1), p.wait_limit));
        if (!ok && lane == 0) report_error(g_status, kErrWaitFull | kKid | (7 << 13));
        ++no_o;
        tc_fence_after();
      }
      const bool seen = row_ok && (!TREE || anc != 0);  // a draft of a broken chain sees nothing
      const bool fix = dirty[no & 1] == no + 1;
      // adds the infinities and NaNs of the V blocks made safe to o's 32 columns from
      // c on. TMEM's instructions want the warp together: so it is brought here, and
      // stores that not all lanes make are predicated.
      auto mend_o = [&](int c, float* o) {
        if (!fix) return;  // all lanes alike
        if (seen) {
          const uint16_t* v =
              static_cast<const uint16_t*>(p.v) + it.tok0 * (TREE ? p.v_seq : p.v_row) + it.g * p.v_head + c;
          for (int i = 0; i < nb; ++i) {
            const int kb = it.b0 + (solo ? 2 * i + slot : i);
            if (kb < fix0) continue;
            for (int key = kb * kRows; key < min(kb * kRows + kRows, it.kend); ++key) {
              if (!(seen32<TREE>(key, lim, anc) & 1u)) continue;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const uint16_t w = v[key * p.v_row + e];
                if (nonfinite<BF16>(w)) o[e] += widen<BF16>(w);
              }
            }
          }
        }
        __syncwarp();
      };
      auto load_o = [&](int c, float* o) {
        tmem_ld32(o_addr + c, o);
        tmem_wait_ld<32>(o);
        mend_o(c, o);
      };
      if (ok && warp_ok && !joined) {
        if (nb > 0) {
          const float inv = !seen ? 0.f : l != 0.f ? 1.0f / l : NAN;  // all scores -inf: 0 / 0
          uint16_t* out = static_cast<uint16_t*>(p.out) + it.tok0 * (TREE ? p.o_seq : p.o_tok) + tok * p.o_tok +
                          (it.g * p.group + row_head) * p.o_head;
          uint32_t odds[2] = {0, 0};  // NaN where a result of the row is not finite
          if (HD == 128 && p.wide_out) {
            // A thread has a row, and 32 rows are 32 lines a store. So the rounded
            // row goes back to TMEM, over columns of o already read, and comes out
            // four lanes to a row, 32 bytes each: eight whole lines a store (7 prompts
            // up to 1024, 32/8 heads of 128: 21.5 us so, 22.3 row by row; of 8184
            // tokens 374 and 377; rows of 64, 30.5 and 30.0, stay as they are).
            const unsigned long long mine = row_ok ? reinterpret_cast<unsigned long long>(out) : 0;
            uint16_t* to[4];  // rows 8i + lane / 4
#pragma unroll
            for (int i = 0; i < 4; ++i) to[i] = reinterpret_cast<uint16_t*>(__shfl_sync(0xffffffffu, mine, 8 * i + (lane >> 2)));
#pragma unroll 1
            for (int c = 0; c < HD; c += 64) {
              uint32_t w[32];  // word 8q + 2i + e of the row's 32, which lane q of four gets as its (2i + e)th
              float o[64];
              tmem_ld32(o_addr + c, o);
              tmem_ld32(o_addr + c + 32, o + 32);
              tmem_wait_ld<64>(o);
              mend_o(c, o);
              mend_o(c + 32, o + 32);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                w[k % 8 / 2 * 8 + k / 8 * 2 + k % 2] = seen ? pack16<BF16>(o[2 * k] * inv, o[2 * k + 1] * inv) : 0u;
#pragma unroll
              for (int k = 0; k < 32; ++k) odds[k & 1] = probe<BF16>(w[k], odds[k & 1]);
              tmem_st16(o_addr + c, w);
              tmem_st16(o_addr + c + 16, w + 16);
              tmem_wait_st();
              __syncwarp();
#pragma unroll
              for (int h = 0; h < 2; ++h) tmem_ld_quads(o_addr + (static_cast<uint32_t>(16 * h) << 16) + c, w + 16 * h);
              tmem_wait_ld<32>(reinterpret_cast<float*>(w));
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = w[i / 2 * 16 + e / 2 * 4 + i % 2 * 2 + e % 2];
                st_global32(to[i] != nullptr, to[i] + c + 16 * (lane & 3), x);
              }
            }
          } else {
            // a thread writes its row, 32 bytes at a time where out is so aligned
#pragma unroll 1
            for (int c = 0; c < HD; c += 32) {
              float o[32];
              load_o(c, o);
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = seen ? pack16<BF16>(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
              if (HD == 64 && p.wide_out) {
                st_global32(row_ok, out + c, w);
                st_global32(row_ok, out + c + 16, w + 8);
              } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) st_global16(row_ok, out + c + u * 8, w + 4 * u);
              }
#pragma unroll
              for (int e = 0; e < 16; ++e) odds[e & 1] = probe<BF16>(w[e], odds[e & 1]);
            }
          }
          bool odd = false;
#pragma unroll
          for (int k = 0; k < 2; ++k) odd |= wild<BF16>(odds[k]);
          if (odd && seen && inv == inv) {
            if (TREE) again = true;
            else settle<BF16, HD, TREE>(p, it, lim, anc, out, 0, 1);
          }
        }
      } else if (TREE && joined) {
        // the ring is free once the other slot's products are done too
        if (ok && blocks_of(it, slot ^ 1) > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(&ofull[slot ^ 1], 0, p.wait_limit));
          if (!ok && lane == 0) report_error(g_status, kErrWaitFull | kKid | (9 << 13));
        }
        const bool here = ok && warp_ok && nb > 0;  // this warp has sums
        const float2 ml = !seen ? ml_of_nothing() : nb > 0 ? make_float2(-neg, l) : ml_without_keys();
        if (!solo) {
          join_ml[slot * kRows + r] = ml;
          if (here) {
#pragma unroll 1
            for (int c = 0; c < HD; c += 32) {
              float o[32];
              load_o(c, o);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                join_o[(slot * (HD / 4) + c / 4 + e) * kRows + r] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
          }
        } else {
          // each slot joins one half of the columns and hands the other half over
          swap_ml[slot * kRows + r] = ml;
          const int mine = slot * (HD / 2), other = HD / 2 - mine;
          if (here) {
#pragma unroll 1
            for (int c = 0; c < HD / 2; c += 32) {
              float o[32];
              load_o(other + c, o);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                swap_o[((other + c) / 4 + e) * kRows + r] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
          }
          named_bar_sync(1, 256);
          const float2 to = swap_ml[(slot ^ 1) * kRows + r];
          const float top = fmaxf(ml.y != 0.f ? ml.x : -INFINITY, to.y != 0.f ? to.x : -INFINITY);
          const float fm = weight_of(ml, top), ft = weight_of(to, top);
          const bool has = has_o(ml), other_has = has_o(to);
          if (slot == 0) {
            const float sum = fm * ml.y + ft * to.y;
            join_ml[r] = sum != 0.f ? make_float2(top, sum) : !seen ? ml : make_float2(has || other_has ? 0.f : -INFINITY, 0.f);
          }
          if (ok && warp_ok) {
#pragma unroll 1
            for (int c = 0; c < HD / 2; c += 32) {
              float o[32];
              if (nb > 0) load_o(mine + c, o);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int at = ((mine + c) / 4 + e) * kRows + r;
                float4 x = other_has ? swap_o[at] : make_float4(0.f, 0.f, 0.f, 0.f);
                x.x = has ? fmaf(fm, o[4 * e], ft * x.x) : ft * x.x;
                x.y = has ? fmaf(fm, o[4 * e + 1], ft * x.y) : ft * x.y;
                x.z = has ? fmaf(fm, o[4 * e + 2], ft * x.z) : ft * x.z;
                x.w = has ? fmaf(fm, o[4 * e + 3], ft * x.w) : ft * x.w;
                join_o[at] = x;
              }
              __syncwarp();
            }
          }
        }
      }
      tc_fence_before();  // O has been read before the next item's first P allows its P.V
      through_with(no);
    }
  }

  if (TREE && joined) {
    // every CTA of the cluster joins its share of the columns
    __syncwarp();
    cluster_sync();
    if (warp < 8) {
      const Item& it = items[0];
      const int half = tid >> 7, r = tid & 127, tile = solo ? 0 : half;
      const int tok = it.t0 + tile * p.tpt + r / p.group;
      if (r / p.group < p.tpt && tok < it.len) {
        const uint32_t ml_at = smem_u32(join_ml + tile * kRows + r), o_at = smem_u32(join_o + tile * (HD / 4) * kRows + r);
        uint16_t* out = static_cast<uint16_t*>(p.out) + it.tok0 * p.o_seq + tok * p.o_tok +
                        (it.g * p.group + r % p.group) * p.o_head;
        const int u0 = blockIdx.x % p.cluster + (solo ? half * p.cluster : 0), step = solo ? 2 * p.cluster : p.cluster;
        switch (p.cluster) {
          case 1: again = join_row<BF16, HD, 1>(ml_at, o_at, out, u0, step); break;
          case 2: again = join_row<BF16, HD, 2>(ml_at, o_at, out, u0, step); break;
          case 4: again = join_row<BF16, HD, 4>(ml_at, o_at, out, u0, step); break;
          case 8: again = join_row<BF16, HD, 8>(ml_at, o_at, out, u0, step); break;
          default: again = join_row<BF16, HD, 16>(ml_at, o_at, out, u0, step); break;
        }
      }
    }
    __syncwarp();
    cluster_sync();  // the cluster's shared memory has been read
  }
  if (TREE && __builtin_expect(again, 0)) {
    // a thread has the row here, and its warp the parents, that it had in its softmax
    const Item& it = items[0];
    const int half = tid >> 7, r = tid & 127, tok = it.t0 + (solo ? 0 : half * p.tpt) + r / p.group;
    uint16_t* out = static_cast<uint16_t*>(p.out) + it.tok0 * p.o_seq + tok * p.o_tok + (it.g * p.group + r % p.group) * p.o_head;
    const int u0 = joined ? blockIdx.x % p.cluster + (solo ? half * p.cluster : 0) : 0;
    settle<BF16, HD, TREE>(p, it, p.pos[it.s] - 1, tree_mask(parents + warp * kTreeMax, tok), out, u0,
                           joined ? (solo ? 2 * p.cluster : p.cluster) : 1);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <bool BF16, int HD, bool TREE>
cudaError_t prepare_t() {
  auto kern = tile_attn_kernel<BF16, HD, TREE>;
  static std::atomic<int> smem_set[kMaxDevices];
  cudaError_t e = set_smem_attr(kern, Shape<HD>::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  // the register split draws on what the block is launched with
  static const int regs = [&] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess ? a.numRegs : 0;
  }();
  return regs == kLaunchRegs ? cudaSuccess : cudaErrorInvalidKernelImage;
}

// attr: two attributes; a cluster of 1 is none.
template <int HD>
cudaLaunchConfig_t config_of(int cluster, long long ctas, cudaStream_t s, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<HD>::kSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = cluster > 1 || ctas <= kEarlyCtas;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cfg;
}

// Clusters of 2^i CTAs that run at once on the current device (0: none do).
template <bool BF16, int HD>
cudaError_t active_t(const int** out) {
  static std::mutex mu;
  static int active[kMaxDevices][kClusterSizes];
  static bool known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!known[dev]) {
    auto kern = tile_attn_kernel<BF16, HD, true>;
    if ((e = prepare_t<BF16, HD, true>()) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
    for (int i = 0; i < kClusterSizes; ++i) {
      cudaLaunchAttribute attr[2];
      cudaLaunchConfig_t cfg = config_of<HD>(1 << i, 1 << i, nullptr, attr);
      cfg.attrs = attr + 1;  // the cluster alone
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&active[dev][i], kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        active[dev][i] = 0;
      }
    }
    known[dev] = true;
  }
  *out = active[dev];
  return cudaSuccess;
}

template <bool BF16, int HD>
cudaError_t launch_prompt_t(const TileAttnParams& p, long long ctas, cudaStream_t s) {
  const cudaError_t e = prepare_t<BF16, HD, false>();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config_of<HD>(1, ctas, s, attr);
  return cudaLaunchKernelEx(&cfg, tile_attn_kernel<BF16, HD, false>, p);
}

template <bool BF16, int HD>
cudaError_t launch_tree_t(const TileAttnParams& p, long long ctas, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config_of<HD>(p.cluster, ctas, s, attr);
  return cudaLaunchKernelEx(&cfg, tile_attn_kernel<BF16, HD, true>, p);
}

}  // namespace

// Sequences longest first: their positions in p.len / p.pos / p.tok0 move.
static void longest_first(TileAttnParams& p, const int* keys) {
  int order[kOpSeqs], tok0[kOpSeqs], len[kOpSeqs], pos[kOpSeqs];
  for (int s = 0; s < p.n_seqs; ++s) order[s] = s, tok0[s] = p.tok0[s], len[s] = p.len[s], pos[s] = p.pos[s];
  std::sort(order, order + p.n_seqs, [&](int a, int b) { return keys[a] != keys[b] ? keys[a] > keys[b] : a < b; });
  for (int s = 0; s < p.n_seqs; ++s) p.tok0[s] = tok0[order[s]], p.len[s] = len[order[s]], p.pos[s] = pos[order[s]];
}

// Work items of a prompt launch: sequences longest first, each from its last
// tokens (which see the most keys) to its first, so that the launch ends on
// small items.
long long tile_prompt_plan(TileAttnParams& p) {
  int keys[kOpSeqs];
  for (int s = 0; s < p.n_seqs; ++s) keys[s] = p.len[s];
  longest_first(p, keys);
  p.tpt = kRows / p.group;
  long long items = 0;
  for (int s = 0; s < p.n_seqs; ++s) {
    p.item0[s] = static_cast<int>(items);
    items += (p.len[s] + 2 * p.tpt - 1) / (2 * p.tpt);
  }
  return items * p.nkv;
}

cudaError_t launch_tile_prompt(const TileAttnParams& p, long long ctas, bool bf16, int hd, cudaStream_t s) {
  if (bf16) return hd == 128 ? launch_prompt_t<true, 128>(p, ctas, s) : launch_prompt_t<true, 64>(p, ctas, s);
  return hd == 128 ? launch_prompt_t<false, 128>(p, ctas, s) : launch_prompt_t<false, 64>(p, ctas, s);
}

static long long blocks_of(const TileAttnParams& p, int s) {
  return p.len[s] ? (p.pos[s] + p.len[s] + kRows - 1) / kRows : 0;
}

// Work items of a tree launch: one cluster per (sequence, pair of tiles, kv
// head), which shares out the sequence's key blocks. The cluster's size is the
// one with the shortest modelled time in units of an iteration (a block, or a
// solo tile's two): the longest CTA, two in a row, or all clusters' work over
// those that run at once, whichever is most; a CTA costs about kStart of them to
// start and finish, and kJoin more where it is joined. The smaller of two that
// are level.
cudaError_t tile_tree_plan(TileAttnParams& p, bool bf16, int hd, long long* ctas) {
  constexpr long long kStart = 2, kJoin = 2;
  p.tpt = kRows / p.group;
  int blocks[kOpSeqs], most_rows = 0;
  for (int s = 0; s < p.n_seqs; ++s) {
    p.tok0[s] = s;
    most_rows = std::max(most_rows, p.len[s]);
    blocks[s] = p.len[s] ? (p.pos[s] + p.len[s] + kRows - 1) / kRows : 0;
  }
  longest_first(p, blocks);
  p.solo = most_rows <= p.tpt;
  long long clusters = 0;
  for (int s = 0; s < p.n_seqs; ++s) {
    p.item0[s] = static_cast<int>(clusters);
    clusters += p.len[s] == 0 ? 0 : p.solo ? 1 : (p.len[s] + 2 * p.tpt - 1) / (2 * p.tpt);
  }
  *ctas = 0;
  if (clusters == 0) return cudaSuccess;
  const int* active = nullptr;
  const cudaError_t e = bf16 ? (hd == 128 ? active_t<true, 128>(&active) : active_t<true, 64>(&active))
                             : (hd == 128 ? active_t<false, 128>(&active) : active_t<false, 64>(&active));
  if (e != cudaSuccess) return e;
  long long best = -1;
  for (int i = 0; i < kClusterSizes; ++i) {
    if (active[i] < 1) continue;
    const int size = 1 << i;
    const long long fixed = kStart + (p.solo || size > 1 ? kJoin : 0);
    // clusters come longest first: past the first `active` of them, one runs
    // behind another of at least its own length
    long long total = 0, longest = 0, seen = 0, second = 0;
    for (int s = 0; s < p.n_seqs; ++s) {
      if (!p.len[s]) continue;
      const int share = p.solo ? 2 * size : size;
      const long long each = (blocks_of(p, s) + share - 1) / share + fixed;
      const long long n = ((s + 1 < p.n_seqs ? p.item0[s + 1] : clusters) - p.item0[s]) * p.nkv;
      longest = std::max(longest, each);
      total += n * each;
      if (seen <= active[i] && seen + n > active[i]) second = 2 * each;
      seen += n;
    }
    const long long cost = std::max(std::max(longest, second), (total + active[i] - 1) / active[i]);
    if (best < 0 || cost < best) {
      best = cost;
      p.cluster = size;
    }
  }
  if (best < 0) return cudaErrorInvalidConfiguration;
  *ctas = clusters * p.nkv * p.cluster;
  return cudaSuccess;
}

cudaError_t launch_tile_tree(const TileAttnParams& p, long long ctas, bool bf16, int hd, cudaStream_t s) {
  if (bf16) return hd == 128 ? launch_tree_t<true, 128>(p, ctas, s) : launch_tree_t<true, 64>(p, ctas, s);
  return hd == 128 ? launch_tree_t<false, 128>(p, ctas, s) : launch_tree_t<false, 64>(p, ctas, s);
}

cudaError_t tile_attn_status(int* status, cudaStream_t s) {
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  e = cudaMemcpyFromSymbol(status, g_status, 2 * sizeof(int));
  if (e != cudaSuccess || (!status[0] && !status[1])) return e;
  const int zero[2] = {0, 0};
  return cudaMemcpyToSymbol(g_status, zero, sizeof zero);
}

}  // namespace lps
