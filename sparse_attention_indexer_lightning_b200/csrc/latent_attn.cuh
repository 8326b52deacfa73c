// Attention of query tokens over whole spans of the latent cache on the
// tensor cores (tcgen05): the window form (the first n_sink rows of a sequence
// plus a sliding or block-aligned window of the latest ones; the sinks and the
// window of "Latent Sparse Attention", "The method, term by term", step 6) and
// the tree form (a context and, behind it, drafted rows of which a token sees
// its own branch).  A latent row is 576 bf16 elements, the key of every head;
// its first 512 are the value (absorbed MLA, as in sparse_attn.cuh):
//
//   z(s) = scale * q . c[s],  lse = log sum_s exp z(s),  o = sum_s exp(z(s) - lse) c[s, :512]
//
// The query heads of a sequence's tokens are consecutive rows of q, so 128 of
// them (whatever the number of heads) are the M of every MMA.  One pass over
// the rows any of them sees, in tiles of 128, with the running maximum and sum
// of the softmax.
//
// Two CTAs of a cluster share the 128 query rows (tcgen05 cta_group::2, M =
// 128): CTA c holds query rows 64c .. 64c + 63, their logits and their fp32
// output of all 512 value columns.  An accumulator of 64 rows x N columns lies
// in 128 lanes x N / 2 tensor-memory columns (lane r and lane r + 64 hold row
// r's first and second half), so the output takes 256 of the 512 columns and
// two tiles' logits 128.  (One CTA with all 128 rows would need all 512 for
// its output, and two CTAs with half of the value columns each would both
// compute the logits: 1664 against 1088 multiply-adds per query row and cache
// row; that form took 2600 cycles per 64 rows, this one needs 2180 per 128.)
// Per tile each CTA stages
//  - half of the rows as keys (64 x 576, 72 KB, in three groups of three
//    panels that are free again as soon as the logits passed them),
//  - half of the value columns of all rows (128 x 256, 64 KB, in two groups,
//    one per output MMA of N = 256),
// and the tensor core of each reads both CTAs' halves.  72 KB of query rows
// and 16 KB of weights fill the shared memory.
//
//  - the first CTA of the pair issues all MMAs, the logits' from one warp and
//    the output's from another (one warp for both spent 800 cycles a tile in
//    its waits); both CTAs' copies report to its barriers;
//  - two tiles' logits are in flight, so the softmax of a tile runs beside the
//    MMAs of its neighbours;
//  - a row's logits of a tile lie in two lanes, so two threads share a row
//    and exchange its maximum; the weights go to shared memory as bf16;
//  - the output is rescaled only when a row's maximum grew by more than 16
//    (in log2 units: weights stay below 2^16, which neither bf16 nor fp32
//    holds less exactly than weights below 1); the sinks, a few rows, come
//    after the window, so that the first reference is the maximum of many.
//
// Rounding to fewer bits: the weights (bf16, half a step is 2^-8 of a weight;
// the sum that divides the output is that of the rounded weights, so they
// still sum to 1) and the output when it is asked for in bf16.  Logits, sums,
// lse are fp32.
//
// Masked places weigh exactly 0 whatever they hold: a tile that not every row
// sees whole is checked for logits that are not finite, and only then the
// staged values are searched for elements that are not finite (a weight of 0
// times one of them would be NaN) and cleared.  A visible row with a NaN or
// +inf logit makes its own query row NaN, and no other.  A visible logit of
// -inf weighs 0, and 0 times a value that is not finite is NaN: a whole tile's
// MMA gives that in the value's column, and of a cleared tile the rows in
// question are looked at in the cache and make the whole query row NaN.
//
// Query rows that would leave pairs idle (few of them over a long span, or
// sequences of very different lengths): the tiles of all of them, laid out one
// after another, are cut into equal runs, one per pair (LaIter).  An item that
// a cut goes through is written in parts (fp32, with their lse) to the
// workspace, at most two parts a pair, and latent_attn_combine_kernel joins
// them.
//
// Measured on a B200 (GPU time after a rest, below the power cap): 4096 tokens
// x 128 heads over 4 + 512 rows 779 us (756 TFLOP/s); 16 drafted tokens x 128
// heads over 32768 rows 138 us with the join (1.06 PFLOP/s; a tile about 4000
// cycles, the four softmax steps of a row in a chain, where its MMAs take
// 2180); 64 single tokens x 128 heads 22 us.

#pragma once

#include "common.cuh"
#include "sparse_attn.cuh"

namespace lsi {

constexpr int kLaRows = 128;                          // query rows of a CTA pair: the MMAs' M
constexpr int kLaHalf = 64;                           // ... of a CTA
constexpr int kLaTile = 128;                          // cache rows per tile
constexpr int kLaFew = 32;                            // a tile of at most so many rows is staged as so many
constexpr int kLaPanels = kAttnLatent / 64;           // 9 panels of 64 elements
constexpr int kLaKGroups = 3, kLaKPer = 3;            // the key panels' groups
constexpr int kLaPanelBytes = kLaHalf * 128;          // 8 KB: 64 elements of 64 rows
constexpr int kLaVGroup = 2 * kLaTile * 128;          // 32 KB: two value panels of 128 rows
// items and query and key copies, logit MMAs, output MMAs, 4 softmax and epilogue, value copies
constexpr int kLaThreads = 8 * 32;
constexpr int kLaColO = 0, kLaColS = 256;             // tensor-memory columns
constexpr float kLaLazy = 16.f;                       // log2 growth of a maximum that forces a rescale
// An item's own cost in tiles: its query, its output.  Of 1 to 5 in cut batches of long and short contexts, 2 took 2 to
// 4 percent longer than 3, and 4 as long as 3, but 4 also cuts 5 tokens over 100 rows (17 us for 14).
constexpr int kLaItemCost = 3;

// First row of the window of the token at position p.
__host__ __device__ inline int la_window_lo(int p, int window, int align) {
  if (window <= 0) return 0;
  const int x = p - window + 1;
  return x <= 0 ? 0 : x - x % align;
}

__device__ __forceinline__ uint64_t la_low_mask(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// The rows that a tile of query rows can see, cut into tiles of 128.
struct LaSpan {
  int sink_len;          // rows [0, sink_len): sinks apart from the window
  int lo, hi;            // window / context rows
  int drafted;           // drafted rows behind the context
  int n0, n1, n2;        // tiles of each
  int lo_max, hi_min;    // rows [lo_max, hi_min) are in every query row's window
  __device__ __forceinline__ int tiles() const { return n0 + n1 + n2; }
  // whether every query row sees all of the tile
  __device__ __forceinline__ bool whole(int kind, int a, int cnt, int n_sink) const {
    return kind == 0 && cnt == kLaTile && a + kLaTile <= hi_min && (a + kLaTile <= n_sink || a >= lo_max);
  }
  // kind 0: rows a .. a + cnt of the sequence; 1: drafted rows a .. a + cnt
  __device__ __forceinline__ void tile(int i, int& kind, int& a, int& cnt) const {
    kind = 0;
    if (i < n1) {
      a = lo + kLaTile * i;
      cnt = hi - a;
    } else if (i < n0 + n1) {
      a = kLaTile * (i - n1);
      cnt = sink_len - a;
    } else {
      kind = 1;
      a = kLaTile * (i - n0 - n1);
      cnt = drafted - a;
    }
    cnt = cnt < kLaTile ? cnt : kLaTile;
  }
};

// One unit of work: a tile of 128 query rows of a sequence over the tiles that they see, or a part of these.
struct LaItem {
  int part;                // its place among the parts, -1: whole
  int t0, n;               // the sequence's first token and number of tokens
  int r0, grow0;           // first query row in the sequence, in q (T * H < 2^31)
  int nrows;               // query rows (at most 128)
  int kv, avail;           // rows of the sequence, those that the cache holds (with the drafted ones)
  int row0, rowd;          // cache rows of its row 0 and of its first drafted row (n_rows + T < 2^31)
  LaSpan sp;
  int i0, nt;              // tiles i0 .. i0 + nt - 1; nt < 0: there are no more items
};
constexpr int kLaItems = 3;   // items in shared memory: the copies' warp writes them, the other roles read them

struct LaBars {
  uint64_t qfull, k_full[3], v_full[2];   // first CTA: both CTAs' query rows, key groups, value groups have landed
  uint64_t q_empty, k_empty[3], v_empty[2];   // query rows, key groups, value groups are read
  uint64_t v_seen;                   // the values of a tile that is not whole have landed in both CTAs
  uint64_t sfull[2];                 // logits in tensor memory
  uint64_t s_empty[2];               // first CTA: both CTAs have read them (8 warps)
  uint64_t pfull;                    // first CTA: both CTAs' weights in shared memory (8 warps)
  uint64_t odone;                    // output MMAs of a tile are complete
  uint64_t mx[2];                    // the two warps that share 32 rows have written their maxima
  uint64_t item_full[kLaItems], item_empty[kLaItems];
  uint64_t drain[2];                 // all MMAs of an issuing warp are complete
  uint32_t tmem_base;
  int abort_flag;
  int idle;                          // cut form: the pair has no places
  LaItem item[kLaItems];
};
constexpr size_t kLaOffK = size_t(kLaPanels) * kLaPanelBytes;               // behind the query rows
constexpr size_t kLaOffV = kLaOffK + size_t(kLaPanels) * kLaPanelBytes;
constexpr size_t kLaOffP = kLaOffV + 2 * size_t(kLaVGroup);
constexpr size_t kLaOffX = kLaOffP + 2 * size_t(kLaPanelBytes);             // exchanged maxima: 2 x 128 floats
constexpr size_t kLaOffL = kLaOffX + 2 * 128 * sizeof(float);               // exchanged sums: 128 + 64 floats
constexpr size_t kLaOffBars = kLaOffL + 192 * sizeof(float);
constexpr size_t kLaSmem = kLaOffBars + 640;
static_assert(sizeof(LaBars) <= 640, "barrier block");
static_assert(kLaSmem <= 232448, "shared memory budget");
struct LatentAttnParams {
  const uint16_t* q = nullptr;        // [T * H][576]
  const uint16_t* latent = nullptr;   // [n_rows][576]
  const int32_t* q_start = nullptr;   // [B + 1]
  const int32_t* kv_len = nullptr;    // [B]: window: rows with the tokens' own; tree: context rows
  const int64_t* row_off = nullptr;   // [B] or nullptr (0)
  const uint64_t* tree = nullptr;     // [T][words] or nullptr: the window form
  int words = 0;
  int B = 0, T = 0, H = 0;
  int max_q = 0, max_tiles = 0;       // tokens of a sequence at most, and their tiles of 128 rows
  int64_t n_rows = 0;
  int window = 0, align = 1, n_sink = 0;   // window <= 0 (tree only): the whole context
  float scale = 0.f;
  int pairs = 1;                      // CTA pairs of the grid
  int cut = 0;                        // equal runs of tiles per pair; else whole items in turn
  int out_bf16 = 0;
  void* out = nullptr;                // [T * H][512]
  float* lse = nullptr;               // [T * H] or nullptr
  // cut form: pair p's part of the item that its run begins inside of (2 p) and that it ends inside of (2 p + 1)
  float* part_o = nullptr;            // [2 * pairs][128][512]
  float* part_lse = nullptr;          // [2 * pairs][128]
  struct LaJoin* joins = nullptr;     // [pairs]
};

// The item that pair p's run ends inside of, if it begins there too: its first row, its rows, and how many pairs have
// a part of it (0: there is none).
struct LaJoin {
  int64_t row0;
  int nrows, parts;
};

// Box of 64 elements x rows x panels (y the row, z the panel) into this CTA's shared memory, reported to a barrier
// of the pair (a cluster address).
__device__ __forceinline__ void la_load_3d(void* dst, const CUtensorMap* map, uint32_t bar, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(y), "r"(z)
      : "memory");
}

// After an abort: the copies in flight (microseconds) land before the CTA ends.
__device__ __forceinline__ void la_settle() {
  const uint64_t t = globaltimer_ns();
  while (globaltimer_ns() - t < 1000000ull) __nanosleep(1000);
}

// Rows of a tile as it is staged.
__device__ __forceinline__ int la_box_rows(int cnt) { return cnt <= kLaFew ? kLaFew : kLaTile; }

// Warp-uniform bounded wait of lane 0.  What the other lanes do in shared memory behind it is kept there: by a compiler
// barrier where they write (the vote holds them until lane 0 has seen the phase), by a warp barrier, which also orders
// memory, where they read what other warps wrote (la_wait_read; without it they met the old values now and then).
__device__ __forceinline__ bool la_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  const bool ok = warp_wait<false>(bar, parity, abort_flag);
  asm volatile("" ::: "memory");
  return ok;
}
__device__ __forceinline__ bool la_wait_read(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  const bool ok = warp_wait<false>(bar, parity, abort_flag);
  __syncwarp();
  return ok;
}

// Warp-uniform bounded wait in which every lane tests the barrier: when the
// phase is complete already, the common case of the MMA warp, it costs one
// test and a vote.
__device__ __forceinline__ bool la_wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return la_wait(bar, parity, abort_flag);
}

// Address of this CTA's shared-memory object in CTA `rank` of the cluster, and an arrival there.  What the arrival
// tells of (logits that have been read, weights behind a proxy fence) concerns the tensor cores alone, so it takes no
// release over the cluster: that, and an acquire fence at the other end, cost 1000 cycles each (10000 cycles a tile).
__device__ __forceinline__ uint32_t la_map(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void la_arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// The arrival, and a test of a phase that is known to be complete, for what the other CTA's warps read themselves:
// ordered over the cluster.
__device__ __forceinline__ void la_arrive_release(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void la_acquire(uint64_t* bar, uint32_t parity) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(parity)
      : "memory");
}
__device__ __forceinline__ void la_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 2^x: the hardware's approximation (relative error 2^-22; 0 below 2^-126).
__device__ __forceinline__ float la_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void la_add2(uint64_t& acc, uint64_t v) {
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(acc) : "l"(v));
}

__device__ __forceinline__ float la_sum2(uint64_t v) {
  float a, b;
  unpack_f32x2(v, a, b);
  return a + b;
}

// One MMA of the CTA pair (K = 16), issued by a converged warp through one elected lane.
__device__ __forceinline__ void la_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The barrier at bar's place receives an arrival once the MMAs issued so far are done, in the CTAs of the mask (by
// default both).
__device__ __forceinline__ void la_commit_both(uint64_t* bar, uint16_t mask = 3) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"(mask)
      : "memory");
}

// Sets the masked places of 32 logits to -inf; whether one of the 32 (stale ones among them) was not finite.
__device__ __forceinline__ bool la_mask_row(uint32_t (&v)[32], uint32_t vis) {
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const uint32_t mag = v[j] & 0x7fffffffu;
    top = top > mag ? top : mag;
    if (!(vis & (1u << j))) v[j] = 0xff800000u;
  }
  return top >= 0x7f800000u;
}

// Rare: whether a lane's query row sees (`vis`: cache row `row0` and the 63 behind it) a cache row with a logit of -inf
// (`low`: its bits before the scale's sign) and a value that is not finite.  Called by a whole warp, whose logits are
// still at `scol`: reading them again keeps 64 comparisons out of the tiles' code.
__device__ __noinline__ bool la_low_rows(const uint16_t* latent, int64_t row0, uint32_t scol, uint64_t vis,
                                         uint32_t low) {
  bool odd = false;
#pragma unroll 1
  for (int h = 0; h < 64; h += 32) {
    uint32_t v[32], mine = 0u;
    tmem_ld_32x32_nowait(scol + h, v);
    tmem_wait_ld(v);
#pragma unroll
    for (int j = 0; j < 32; ++j) mine |= v[j] == low ? 1u << j : 0u;
    mine &= static_cast<uint32_t>(vis >> h);
    for (uint32_t todo = __reduce_or_sync(0xffffffffu, mine); todo; todo &= todo - 1) {
      const int j = __ffs(todo) - 1;
      const uint4* row = reinterpret_cast<const uint4*>(latent + (row0 + h + j) * kAttnLatent);
      bool bad = false;
      for (int c = threadIdx.x & 31; c < kAttnValue / 8; c += 32) {
        const uint4 x = __ldg(row + c);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          bad |= (w[k] & 0x7f80u) == 0x7f80u || (w[k] & 0x7f800000u) == 0x7f800000u;
      }
      if (__any_sync(0xffffffffu, bad)) odd |= (mine >> j) & 1u;
    }
  }
  return odd;
}

// One row's largest logit of a tile in log2 units (masked places hold -inf).
__device__ __forceinline__ float la_row_max(const uint32_t (&va)[32], const uint32_t (&vb)[32], float sl2) {
  float x[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
  for (int j = 0; j < 32; ++j) x[j & 3] = fmaxf(x[j & 3], fmaxf(__uint_as_float(va[j]), __uint_as_float(vb[j])));
  const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
  return top == neg_inf() ? top : sl2 * top;
}

// One row's weights of a tile, packed to bf16 pairs, and their sums: of the weights and of the rounded weights.
// Masked places hold -inf and weigh 0 (sl2 is not 0).
__device__ __forceinline__ void la_row_weights(const uint32_t (&va)[32], const uint32_t (&vb)[32], float sl2,
                                               float ref, uint32_t (&pw)[32], float& l, float& lt) {
  const uint64_t s2 = pack_f32x2(sl2, sl2), r2 = pack_f32x2(-ref, -ref);
  uint64_t a[2] = {0ull, 0ull}, c[2] = {0ull, 0ull};
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    uint64_t z = pack_f32x2(__uint_as_float(e < 16 ? va[2 * e] : vb[2 * e - 32]),
                            __uint_as_float(e < 16 ? va[2 * e + 1] : vb[2 * e - 31]));
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(z) : "l"(s2), "l"(r2));
    float p0, p1;
    unpack_f32x2(z, p0, p1);
    p0 = la_exp2(p0);
    p1 = la_exp2(p1);
    la_add2(a[e & 1], pack_f32x2(p0, p1));
    const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
    pw[e] = *reinterpret_cast<const uint32_t*>(&pb);
    la_add2(c[e & 1], pack_f32x2(__uint_as_float(pw[e] << 16), __uint_as_float(pw[e] & 0xffff0000u)));
  }
  la_add2(a[0], a[1]);
  la_add2(c[0], c[1]);
  l += la_sum2(a[0]);
  lt += la_sum2(c[0]);
}

// 128 bytes of each of a warp's 32 rows, staged with the 16-byte pieces of row i at their place ^ (i & 7), to rows
// `pitch` bytes apart: eight lanes a row, four rows a store.
__device__ __forceinline__ void la_rows_out(const uint8_t* stage, uint8_t* dst, int pitch, uint32_t keep, int lane) {
  __syncwarp();
  const int piece = lane & 7;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int i = 4 * u + (lane >> 3);
    const uint4 v = *reinterpret_cast<const uint4*>(stage + i * 128 + ((piece ^ (i & 7)) << 4));
    if ((keep >> i) & 1u) *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(i) * pitch + 16 * piece) = v;
  }
  __syncwarp();
}

// Tensor maps over rows of 9 panels of 64 elements, boxes of 64 elements x rows x panels, 128-byte swizzle.
struct LaMaps {
  CUtensorMap q;            // q rows: 64 x 3 panels
  CUtensorMap k, v;         // latent rows: 64 x 3, 128 x 2
  CUtensorMap k_few, v_few; // latent rows: 16 x 3, 32 x 2
};

// Query tile `qtile` of sequence b (-1: its last), whole; false where the sequence has none.  `all` is the number of
// query tiles.  Tables that do not hold set the fault word (`tell`: the calling thread does that) and what they name
// wrongly is not seen.
__device__ __forceinline__ bool la_item(const LatentAttnParams& P, int b, int qtile, bool tell, LaItem& w, int& all) {
  const int H = P.H;
  w.t0 = __ldg(P.q_start + b);
  const int t1 = __ldg(P.q_start + b + 1);
  int kv = __ldg(P.kv_len + b);
  const int64_t off = P.row_off ? __ldg(P.row_off + b) : 0;
  if (w.t0 < 0 || t1 < w.t0 || t1 > P.T) {            // not a prefix of the tokens: nothing of it is computed
    if (tell) atomicOr(&g_fault, FAULT_BAD_INDEX);
    return false;
  }
  const int n = w.n = t1 - w.t0;
  const int64_t seq_rows = static_cast<int64_t>(n) * H;
  if (n > P.max_q && tell)
    atomicOr(&g_fault, FAULT_BAD_INDEX);              // more tokens than max_q: those past max_tiles are not computed
  const int tiles = static_cast<int>((static_cast<uint32_t>(seq_rows) + kLaRows - 1) / kLaRows);   // T * H < 2^31
  all = tiles < P.max_tiles ? tiles : P.max_tiles;
  if (qtile < 0) qtile = all - 1;
  if (qtile < 0 || qtile >= all) return false;
  w.r0 = qtile * kLaRows;
  w.nrows = static_cast<int>(seq_rows - w.r0 < kLaRows ? seq_rows - w.r0 : kLaRows);
  w.grow0 = w.t0 * H + w.r0;
  const uint32_t first_row = static_cast<uint32_t>(w.r0);        // T * H < 2^31
  const int tok_first = first_row / static_cast<uint32_t>(H);
  const int tok_last = (first_row + w.nrows - 1) / static_cast<uint32_t>(H);
  const bool is_tree = P.tree != nullptr;
  const int own = is_tree ? n : 0;                    // drafted rows behind kv
  if ((kv < 0 || off < 0 || off > P.n_rows || kv + static_cast<int64_t>(own) > P.n_rows - off) && tell)
    atomicOr(&g_fault, FAULT_BAD_INDEX);              // rows outside the cache are not seen
  w.kv = kv = kv < 0 ? 0 : kv > P.n_rows ? static_cast<int>(P.n_rows) : kv;
  int avail = 0;
  if (off >= 0 && off < P.n_rows)
    avail = static_cast<int>(P.n_rows - off < kv + static_cast<int64_t>(own) ? P.n_rows - off : kv + own);
  w.avail = avail;
  w.row0 = avail > 0 ? static_cast<int>(off) : 0;
  w.rowd = w.row0 + kv;
  LaSpan& sp = w.sp;
  if (is_tree) {
    const int ctx = kv < avail ? kv : avail;
    sp.drafted = avail - ctx < 64 * P.words ? avail - ctx : 64 * P.words;   // rows past the mask's words are not seen
    sp.hi = sp.hi_min = ctx;
    sp.lo = la_window_lo(kv, P.window, P.align);      // a token's depth is 0 at least, n - 1 at most
    sp.lo_max = la_window_lo(kv + n - 1, P.window, P.align);
  } else {
    const int p0 = kv - n + tok_first, p1 = kv - n + tok_last;
    sp.drafted = 0;
    sp.hi = p1 + 1 < avail ? p1 + 1 : avail;
    sp.hi_min = p0 + 1 < avail ? p0 + 1 : avail;
    sp.lo = la_window_lo(p0, P.window, P.align);
    sp.lo_max = la_window_lo(p1, P.window, P.align);
  }
  if (sp.hi < 0) sp.hi = 0;
  sp.sink_len = P.n_sink < sp.hi ? P.n_sink : sp.hi;
  if (sp.lo <= sp.sink_len) {
    sp.lo = 0;
    sp.sink_len = 0;
  }
  sp.n0 = (sp.sink_len + kLaTile - 1) / kLaTile;
  sp.n1 = sp.hi > sp.lo ? (sp.hi - sp.lo + kLaTile - 1) / kLaTile : 0;
  sp.n2 = (sp.drafted + kLaTile - 1) / kLaTile;
  w.part = -1;
  w.i0 = 0;
  w.nt = sp.tiles();
  return true;
}

// The items of a pair, found by the whole warp that hands them out: every sequence has places, laid out one behind
// another.  Lane i holds the places of sequence b0 + i, so that sequences without tokens (a padded batch has many) are
// stepped over 32 at a time.
//
// Whole items: one place per item; pair p takes the places p, p + pairs, ...  (Of one sequence, or as many sequences of
// one item at most as there are pairs, the places are counted without a look at the tables, and some have no item.)
//
// Cut: every sequence's items weigh its last one's tiles and kLaItemCost; of the sum of all, pair p takes the places
// total * p / pairs .. total * (p + 1) / pairs.  Place x of an item is its tile x - kLaItemCost (the first places are
// its own cost; tiles beyond the weight belong to the last place).
struct LaIter {
  int lane, pairs;
  int64_t pos, end, base;                   // next place, end of the pair's, first place of sequence b0
  int64_t total;                            // cut: all places
  int b0, weight;                           // first sequence of the group; places per item of this lane's
  int64_t mine, upto, group;                // places of this lane's sequence, with those before it, of the group
  int64_t item_end;                         // cut: one behind the item's last place
  bool guess;                               // places counted without the tables
  __device__ __forceinline__ void start(const LatentAttnParams& P, LaBars* bars, int lane_) {
    lane = lane_;
    pairs = static_cast<int>(gridDim.x >> 1);
    const int64_t p = blockIdx.x >> 1;
    guess = !P.cut && (P.B == 1 || (P.max_tiles == 1 && P.B <= pairs));
    base = total = item_end = 0;
    pos = p;
    end = INT64_MAX;
    for (b0 = 0;; b0 += 32) {
      load(P);
      total += group;
      if (!P.cut || b0 + 32 >= P.B) break;
    }
    if (!P.cut) return;
    pos = total * p / pairs;
    end = total * (p + 1) / pairs;
    if (lane == 0) bars->idle = pos == end;
    if (b0 > 0) {                           // the first group again
      b0 = -32;
      group = 0;
    }
  }
  __device__ __forceinline__ void load(const LatentAttnParams& P) {
    const int b = b0 + lane;
    mine = 0;
    weight = 1;
    if (b < P.B) {
      LaItem w;
      int all;
      if (guess) {
        mine = P.max_tiles;
      } else if (la_item(P, b, -1, blockIdx.x == 0, w, all)) {
        if (P.cut) weight = w.nt + kLaItemCost;
        mine = static_cast<int64_t>(all) * weight;
      }
    }
    upto = mine;                            // with those before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    group = __shfl_sync(0xffffffffu, upto, 31);
  }
  __device__ __forceinline__ bool next(const LatentAttnParams& P, LaItem& w) {
    while (pos < end) {
      while (pos >= base + group) {
        base += group;
        b0 += 32;
        if (b0 >= P.B) return false;
        load(P);
      }
      const int f = __ffs(__ballot_sync(0xffffffffu, pos - base < upto)) - 1;
      const int64_t first = base + __shfl_sync(0xffffffffu, upto - mine, f);
      const int64_t at = pos - first;
      const int per = P.cut ? __shfl_sync(0xffffffffu, weight, f) : 1;
      const int64_t q = P.cut ? at / per : at;
      int all;
      const bool has = la_item(P, b0 + f, static_cast<int>(q), guess && (blockIdx.x & 1) == 0, w, all);
      if (!P.cut) {
        pos += pairs;
        if (has) return true;
        continue;
      }
      item_end = first + (q + 1) * per;
      const int x0 = static_cast<int>(at - q * per);
      const int x1 = end - pos < per - x0 ? x0 + static_cast<int>(end - pos) : per;
      const int n = w.nt;
      int i0 = x0 - kLaItemCost, i1 = x1 - kLaItemCost;
      i0 = i0 < 0 ? 0 : i0 < n ? i0 : n;
      i1 = x1 == per ? n : i1 < 0 ? 0 : i1 < n ? i1 : n;
      w.i0 = i0;
      w.nt = i1 - i0;
      if (x0 > 0 || x1 < per) w.part = 2 * static_cast<int>(blockIdx.x >> 1) + (x0 > 0 ? 0 : 1);
      pos += x1 - x0;
      return true;
    }
    return false;
  }
};

// Item `ic` of the CTA, copied out of shared memory by a warp, which gives its place back at once.
__device__ __forceinline__ bool la_next_item(LaBars* bars, int ic, LaItem& w, volatile int* abort_flag) {
  const int slot = ic % kLaItems;
  if (!la_wait_read(&bars->item_full[slot], (ic / kLaItems) & 1, abort_flag)) return false;
  w = bars->item[slot];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&bars->item_empty[slot]);
  return true;
}

// Persistent: the roles run through the pair's items (LaIter) at their own pace: the next item's query, first tiles and
// logits are on their way while the output of the last one leaves.  Barrier phases follow counts that run on over the
// items: tiles (g), items with tiles (qn), exchanges (xn).
//
// The order of the roles in the source, which branches are named rare and which short loops are rolled change where the
// tiles' loops lie in the code and nothing else, but over some 60 forms 16 tokens x 128 heads over 32768 rows took 131
// to 164 us and 4096 tokens over a window of 512 rows 748 to 830.  This one had the lowest mean over the cases.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLaThreads, 1)
    latent_attn_kernel(const __grid_constant__ LaMaps M, const __grid_constant__ LatentAttnParams P) {
  extern __shared__ __align__(1024) uint8_t la_raw[];
  uint8_t* smem = la_raw;
  if (smem_u32(smem) & 1023u) {                       // the swizzle needs what the declaration asks for
    if (threadIdx.x == 0) {
      atomicOr(&g_fault, FAULT_WAIT_TIMEOUT);
      if (P.cut && (blockIdx.x & 1) == 0) P.joins[blockIdx.x >> 1] = LaJoin{0, 0, 0};
    }
    return;
  }
  LaBars* bars = reinterpret_cast<LaBars*>(smem + kLaOffBars);
  volatile int* abort_flag = &bars->abort_flag;
  // (broadcasts of what is the same in a warp anyway let the compiler keep it, and the MMAs' operands, uniform: an
  // MMA whose operands move from a lane's registers takes 48 cycles to issue)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const int cr = static_cast<int>(blockIdx.x & 1);    // rank in the pair
  const int H = P.H;
  const bool is_tree = P.tree != nullptr;

  if (threadIdx.x == 0) {
    mbar_init(&bars->qfull, 1);
    mbar_init(&bars->q_empty, 1);
    for (int g = 0; g < kLaKGroups; ++g) {
      mbar_init(&bars->k_full[g], 1);
      mbar_init(&bars->k_empty[g], 1);
    }
    mbar_init(&bars->v_seen, 1);
    for (int g = 0; g < 2; ++g) {
      mbar_init(&bars->v_full[g], 1);
      mbar_init(&bars->v_empty[g], 1);
      mbar_init(&bars->sfull[g], 1);
      mbar_init(&bars->s_empty[g], 8);
      mbar_init(&bars->mx[g], 2);
    }
    mbar_init(&bars->pfull, 8);
    for (int i = 0; i < kLaItems; ++i) {
      mbar_init(&bars->item_full[i], 1);
      mbar_init(&bars->item_empty[i], 7);             // every warp but the one that writes them
    }
    mbar_init(&bars->odone, 1);
    mbar_init(&bars->drain[0], 1);
    mbar_init(&bars->drain[1], 1);
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  LaIter it;
  if (warp == 0) {
    __syncwarp();
    it.start(P, bars, lane);
    if (lane == 0) {
      tma_prefetch_desc(&M.q);
      tma_prefetch_desc(&M.k);
      tma_prefetch_desc(&M.v);
    }
  }
  tc_fence_before();
  __syncthreads();
  la_cluster_sync();                                  // both CTAs' barriers stand before anyone arrives on them
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);

  if (warp >= 3 && warp <= 6) {
    // ------------------------------------------------------------ softmax + epilogue
    const int quad = warp & 3;                        // warps 3-6: tensor-memory lanes 32 * (warp & 3) ..
    const int tl = quad * 32 + lane;                  // tensor-memory lane
    const int r = tl & 63, half = tl >> 6;            // row of this CTA, and which half of a tile's rows
    const int grp = quad & 1;                         // the two warps that share 32 rows
    const int rq = kLaHalf * cr + r;                  // row of the pair
    const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    float* xch = reinterpret_cast<float*>(smem + kLaOffX);
    const uint32_t pfull0 = la_map(&bars->pfull, 0);
    // a pair without a run (fewer places than pairs) may lie between an item's parts: its own is empty
    if (P.cut && cr == 0 && bars->idle)
      P.part_lse[2 * static_cast<int64_t>(blockIdx.x >> 1) * kLaRows + tl] = neg_inf();
    // logits in log2 units; a scale that is not above 0 turns (or clears) the logits first
    const bool turn = !(P.scale > 0.f);
    const float mult = P.scale < 0.f ? -1.f : 0.f;
    const float sl2 = P.scale == 0.f ? 1.f : fabsf(P.scale) * 1.4426950408889634f;
    bool ok = true;
    const uint32_t s_read[2] = {la_map(&bars->s_empty[0], 0), la_map(&bars->s_empty[1], 0)};
    float* xsum = reinterpret_cast<float*>(smem + kLaOffL);
    int g = 0, xn = 0, vn = 0;                        // tiles, exchanges, tiles that are not whole
    for (int ic = 0; ok; ++ic) {
      LaItem w;
      if (!la_next_item(bars, ic, w, abort_flag)) { ok = false; break; }
      const LaSpan& sp = w.sp;
      const int nt = __shfl_sync(0xffffffffu, w.nt, 0);
      if (nt < 0) break;
      const bool live = rq < w.nrows;
      const int tok = (static_cast<uint32_t>(w.r0) + (live ? rq : w.nrows - 1)) / static_cast<uint32_t>(H);
      // this row's visible rows of the sequence: [0, hi) cut by the sinks and the window
      int hi, lo;
      const uint64_t* branch = nullptr;
      if (is_tree) {
        branch = P.tree + static_cast<int64_t>(w.t0 + tok) * P.words;
        int depth = 0;
        if (P.window > 0) {
          for (int c = 0; c < P.words; ++c) depth += __popcll(__ldg(branch + c) & la_low_mask(w.n - 64 * c));
          depth = depth > 0 ? depth - 1 : 0;
        }
        hi = sp.hi;
        lo = la_window_lo(w.kv + depth, P.window, P.align);
      } else {
        const int p = w.kv - w.n + tok;
        hi = p + 1 < w.avail ? p + 1 : w.avail;
        lo = la_window_lo(p, P.window, P.align);
      }
      float m = neg_inf(), l = 0.f, lt = 0.f;           // reference, sum of the weights, of the rounded weights
      for (int i = 0; i < nt && ok; ++i, ++g) {
        const int st = g & 1;
        int kind, a0, cnt0;
        sp.tile(w.i0 + i, kind, a0, cnt0);
        const bool whole = sp.whole(kind, a0, cnt0, P.n_sink);
        // this thread's rows of the tile: `hs` from a on, cnt of them in the tile
        const int hs = la_box_rows(cnt0) / 2;
        const int a = a0 + hs * half;
        const int left = cnt0 - hs * half, cnt = left < 0 ? 0 : left < hs ? left : hs;
        uint64_t vis = ~0ull;
        if (!whole) {
          if (kind == 0)
            vis = la_low_mask(hi - a < cnt ? hi - a : cnt) & (la_low_mask(P.n_sink - a) | ~la_low_mask(lo - a));
          else
            vis = cnt > 0 ? (__ldg(branch + (a >> 6)) >> (a & 63)) & la_low_mask(cnt) : 0ull;
        }
        if (!la_wait(&bars->sfull[st], (g >> 1) & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        uint32_t va[32], vb[32];
        const uint32_t scol = trow + kLaColS + 64 * st;
        tmem_ld_32x32_nowait(scol, va);
        tmem_ld_32x32_nowait(scol + 32, vb);
        tmem_wait_ld(va);
        tmem_wait_ld(vb);
        if (whole) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) la_arrive_at(s_read[st]);
        }
        if (__builtin_expect(turn, 0)) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            va[j] = __float_as_uint(__uint_as_float(va[j]) * mult);
            vb[j] = __float_as_uint(__uint_as_float(vb[j]) * mult);
          }
        }
        if (!whole) {
          bool bad = la_mask_row(va, static_cast<uint32_t>(vis));
          if (hs == kLaHalf) {
            bad |= la_mask_row(vb, static_cast<uint32_t>(vis >> 32));
          } else {                                      // few rows: 16 columns, all among the first
#pragma unroll
            for (int j = 0; j < 32; ++j) vb[j] = 0xff800000u;
          }
          // A cache row that holds something not finite gives every query row of the pair a logit that is not
          // finite, so both CTAs find out (the tile's values have landed after the output before it is complete), and
          // each warp that does clears its CTA's staged values before its own arrival (two warps that clear the same
          // piece store the same bytes).
          if (__builtin_expect(__any_sync(0xffffffffu, bad), 0)) {
            // a weight of 0 times a visible value that is not finite is NaN, as in a whole tile; here the divisor is
            if (la_low_rows(P.latent, static_cast<int64_t>(kind ? w.rowd : w.row0) + a, scol, vis,
                            P.scale < 0.f ? 0x7f800000u : 0xff800000u))
              lt = __uint_as_float(0x7fffffffu);
            if ((i > 0 && !la_wait(&bars->odone, (g - 1) & 1, abort_flag)) ||
                !la_wait_read(&bars->v_seen, vn & 1, abort_flag)) {
              ok = false;
              break;
            }
            la_acquire(&bars->v_seen, vn & 1);
            for (int c = 0; c < 2; ++c) {
              uint4* v4 = reinterpret_cast<uint4*>(smem + kLaOffV + c * kLaVGroup);
              for (int e = lane; e < 2 * 8 * 2 * hs; e += 32) {
                uint4 x = v4[e];
                uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if ((xw[k] & 0x7f80u) == 0x7f80u) xw[k] &= 0xffff0000u;
                  if ((xw[k] & 0x7f800000u) == 0x7f800000u) xw[k] &= 0x0000ffffu;
                }
                v4[e] = x;
              }
            }
          }
        }
        if (!whole) {
          ++vn;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) la_arrive_at(s_read[st]);
        }
        // the row's maximum: this thread's half and, from the other warp of the pair, the other half
        float mt = la_row_max(va, vb, sl2);
        xch[128 * st + tl] = mt;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->mx[grp]);
        if (!la_wait_read(&bars->mx[grp], xn & 1, abort_flag)) { ok = false; break; }
        ++xn;
        mt = fmaxf(mt, xch[128 * st + (tl ^ 64)]);
        const bool grow = mt > m + kLaLazy;             // true at the first visible finite logit
        const float f = grow ? (m == neg_inf() ? 0.f : la_exp2(m - mt)) : 1.f;
        if (grow) m = mt;
        l *= f;
        lt *= f;
        const float ref = m == neg_inf() ? 0.f : m;
        uint32_t pw[32];
        la_row_weights(va, vb, sl2, ref, pw, l, lt);
        if (i > 0) {
          // the output of the tile before is complete: its weights are read and its accumulator may be rescaled
          if (!la_wait(&bars->odone, (g - 1) & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[32];
              tmem_ld_32x32_nowait(trow + kLaColO + 32 * c, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st_32x32(trow + kLaColO + 32 * c, o);
            }
            tmem_wait_st();
          }
        }
        // weights: row r of the K-major panel of 64 cache rows (128-byte swizzle), 8 rows a piece
        uint8_t* prow = smem + kLaOffP + (hs == 64 ? half * kLaPanelBytes : 0) + r * 128;
        if (__builtin_expect(hs == 64, 1)) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(prow + ((c ^ (r & 7)) << 4)) =
                make_uint4(pw[4 * c], pw[4 * c + 1], pw[4 * c + 2], pw[4 * c + 3]);
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            *reinterpret_cast<uint4*>(prow + (((c + 2 * half) ^ (r & 7)) << 4)) =
                make_uint4(pw[4 * c], pw[4 * c + 1], pw[4 * c + 2], pw[4 * c + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) la_arrive_at(pfull0);
      }
      // ------------------------------------------------------------ output
      if (ok && nt > 0) ok = la_wait(&bars->odone, (g - 1) & 1, abort_flag);
      if (ok && nt > 0) {
        // the row's sums: the two threads' halves
        tc_fence_after();
        xsum[tl] = lt;
        if (half) xsum[128 + r] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->mx[grp]);
        ok = la_wait_read(&bars->mx[grp], xn & 1, abort_flag);
        ++xn;
        lt += xsum[tl ^ 64];
        if (!half) l += xsum[128 + r];
      }
      if (ok) {
        // nothing visible (or only -inf logits): the rounded weights' sum is 0 exactly when that of the weights is
        const bool empty = lt == 0.f;
        const float inv = empty ? 0.f : 1.f / lt;
        const int64_t row = static_cast<int64_t>(w.grow0) + rq;
        const bool parts = w.part >= 0;
        const int64_t part_row = static_cast<int64_t>(w.part) * kLaRows + rq;
        if (half == 0 && live) {
          // (a part that saw nothing but such rows is not empty: the join has to read its NaN)
          const float v = empty ? neg_inf() : parts && l == 0.f ? lt : (m + log2f(l)) * 0.6931471805599453f;
          if (parts)
            P.part_lse[part_row] = v;
          else if (P.lse)
            P.lse[row] = v;
        }
        // Rows leave through the warp's 4 KB of the weights' place (free until its next weights), 128 bytes of each of
        // its 32 rows at a time, so that a store covers four rows' whole lines.  Columns 32 c .. of this lane are
        // value columns 256 (c / 4) + 128 half + 32 (c % 4) ...
        const bool wide = parts || !P.out_bf16;
        const uint32_t keep = __ballot_sync(0xffffffffu, live && !(parts && empty));   // an empty part is not read
        const int64_t row0 = (parts ? static_cast<int64_t>(w.part) * kLaRows : static_cast<int64_t>(w.grow0)) +
                             kLaHalf * cr + (quad & 1) * 32;
        uint8_t* dst = parts ? reinterpret_cast<uint8_t*>(P.part_o) : static_cast<uint8_t*>(P.out);
        dst += row0 * (kAttnValue * (wide ? 4 : 2));
        uint8_t* stage = smem + kLaOffP + quad * 4096;
        uint8_t* mine = stage + lane * 128;
        // (rolled loops: this code runs once an item, and what it takes of the instruction cache the tiles' code
        // misses)
#pragma unroll 2
        for (int c = 0; c < 8; ++c) {
          uint32_t x[32];
          if (nt > 0) {
            tmem_ld_32x32_nowait(trow + kLaColO + 32 * c, x);
            tmem_wait_ld(x);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = 0u;
          }
          const int col = 256 * (c >> 2) + 128 * half + 32 * (c & 3);
          // (a row that saw nothing: its weights were 0 and its values finite, so the accumulator is 0)
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * inv);
          if (wide) {                                   // 32 columns are 128 bytes
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(mine + ((k ^ (lane & 7)) << 4)) =
                  make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          } else {                                      // 64 columns are
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t p2[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 h =
                    __floats2bfloat162_rn(__uint_as_float(x[8 * k + 2 * e]), __uint_as_float(x[8 * k + 2 * e + 1]));
                p2[e] = *reinterpret_cast<const uint32_t*>(&h);
              }
              *reinterpret_cast<uint4*>(mine + (((k + 4 * (c & 1)) ^ (lane & 7)) << 4)) =
                  make_uint4(p2[0], p2[1], p2[2], p2[3]);
            }
          }
          if (wide || (c & 1))
            la_rows_out(stage, dst + (wide ? 4 * col : 2 * (col - 32)), kAttnValue * (wide ? 4 : 2), keep, lane);
        }
      }
    }
  } else if (warp == 0) {
    // ------------------------------------------------------------ items, query and key copies
    // Both CTAs copy their own halves; the first CTA's barriers count both (it alone announces the bytes).  All lanes
    // look for the next item, one hands it on and copies.
    const bool first = cr == 0;
    const uint32_t qfull = la_map(&bars->qfull, 0);
    const uint32_t k_full[3] = {la_map(&bars->k_full[0], 0), la_map(&bars->k_full[1], 0), la_map(&bars->k_full[2], 0)};
    int g = 0, qn = 0;
    LaJoin join{0, 0, 0};
    bool ok = true;
    for (int ic = 0;; ++ic) {
      LaItem w;
      if (!it.next(P, w)) w.nt = w.part = -1;
      if (lane == 0) {
        const int slot = ic % kLaItems;
        ok = mbar_wait<false>(&bars->item_empty[slot], ((ic / kLaItems) & 1) ^ 1, abort_flag);
        if (ok) {
          bars->item[slot] = w;
          mbar_arrive(&bars->item_full[slot]);
          if (w.part >= 0 && (w.part & 1)) {          // begins in this run and goes on in the next pairs'
            int64_t k = (blockIdx.x >> 1) + 1;
            while (k < it.pairs && it.total * k / it.pairs < it.item_end) ++k;
            join.row0 = w.grow0;
            join.nrows = w.nrows;
            join.parts = static_cast<int>(k - (blockIdx.x >> 1));
          }
        }
        if (ok && w.nt > 0) ok = mbar_wait<false>(&bars->q_empty, (qn & 1) ^ 1, abort_flag);
        if (ok && w.nt > 0) {
          ++qn;
          if (first) mbar_arrive_expect_tx(&bars->qfull, 2 * kLaPanels * kLaPanelBytes);
#pragma unroll 1
          for (int c = 0; c < kLaKGroups; ++c)
            la_load_3d(smem + c * kLaKPer * kLaPanelBytes, &M.q, qfull, w.grow0 + kLaHalf * cr, kLaKPer * c);
          for (int i = 0; i < w.nt && ok; ++i) {
            int kind, a, cnt;
            w.sp.tile(w.i0 + i, kind, a, cnt);
            const int box = la_box_rows(cnt) / 2;     // this CTA's half of the rows
            const int row = (kind ? w.rowd : w.row0) + a + box * cr;
#pragma unroll
            for (int c = 0; c < kLaKGroups; ++c) {
              if (!mbar_wait<false>(&bars->k_empty[c], ((g + i) & 1) ^ 1, abort_flag)) { ok = false; break; }
              if (first) mbar_arrive_expect_tx(&bars->k_full[c], 2 * kLaKPer * box * 128);
              la_load_3d(smem + kLaOffK + c * kLaKPer * kLaPanelBytes, box == kLaHalf ? &M.k : &M.k_few, k_full[c], row,
                         kLaKPer * c);
            }
          }
          g += w.nt;
        }
      }
      if (w.nt < 0 || !__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
    }
    if (lane == 0) {
      if (P.cut && first) P.joins[blockIdx.x >> 1] = join;
      if (!ok) la_settle();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ logit MMAs of the pair (first CTA)
    const uint32_t base = smem_u32(smem);
    const uint64_t qdesc = sw128_kmajor_desc(base), kdesc = sw128_kmajor_desc(base + static_cast<uint32_t>(kLaOffK));
    bool ok = true;
    int g = 0, qn = 0;
    for (int ic = 0; ok; ++ic) {
      LaItem w;
      if (!la_next_item(bars, ic, w, abort_flag)) { ok = false; break; }
      const int nt = __shfl_sync(0xffffffffu, w.nt, 0);
      if (nt < 0) break;
      if (nt == 0 || cr == 1) continue;               // the first CTA issues for both
      if (!la_wait_all(&bars->qfull, qn & 1, abort_flag)) { ok = false; break; }
      ++qn;
      for (int i = 0; i < nt; ++i, ++g) {
        int kind, a, cnt;
        w.sp.tile(w.i0 + i, kind, a, cnt);
        const bool full = __shfl_sync(0xffffffffu, la_box_rows(cnt), 0) == kLaTile;
        const uint32_t d = tmem + kLaColS + 64 * (g & 1);
        if (!la_wait_all(&bars->s_empty[g & 1], ((g >> 1) & 1) ^ 1, abort_flag)) { ok = false; break; }
        // the two sizes apart, so that a descriptor is a constant away from one per group; loops over the groups, for
        // the instruction cache's sake
#pragma unroll 1
        for (int c = 0; c < kLaKGroups; ++c) {
          if (!la_wait_all(&bars->k_full[c], g & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint64_t qd = qdesc + c * (kLaKPer * kLaPanelBytes / 16);
          const uint64_t kd = kdesc + c * (kLaKPer * kLaPanelBytes / 16);
          const uint32_t acc0 = c ? 1u : 0u;
          if (full) {
#pragma unroll
            for (int p = 0; p < kLaKPer; ++p)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                la_mma(d, qd + (p * kLaPanelBytes + 32 * kk) / 16, kd + (p * kLaPanelBytes + 32 * kk) / 16,
                       idesc_bf16_f32(kLaRows, kLaTile), (p | kk) ? 1u : acc0);
          } else {
            // few rows: a group's panels lie 16 rows apart
#pragma unroll
            for (int p = 0; p < kLaKPer; ++p)
#pragma unroll 1
              for (int kk = 0; kk < 4; ++kk)
                la_mma(d, qd + (p * kLaPanelBytes + 32 * kk) / 16, kd + (p * (kLaFew * 64) + 32 * kk) / 16,
                       idesc_bf16_f32(kLaRows, kLaFew), (p | kk) ? 1u : acc0);
          }
          la_commit_both(&bars->k_empty[c]);
        }
        if (!ok) break;
        la_commit_both(&bars->sfull[g & 1]);
        if (i == nt - 1) la_commit_both(&bars->q_empty);
      }
    }
    // all MMAs this warp started are complete once `drain` flips
    if (cr == 0 && qn > 0) {
      la_commit_both(&bars->drain[0], 1);
      if (lane == 0) mbar_wait_drain(&bars->drain[0], 0);
      __syncwarp();
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ output MMAs of the pair (first CTA)
    const uint32_t base = smem_u32(smem);
    constexpr uint32_t idesc_o = idesc_bf16_f32(kLaRows, 256) | (1u << 16);   // B MN-major
    const uint64_t pdesc = sw128_kmajor_desc(base + static_cast<uint32_t>(kLaOffP)),
                   vdesc = sw128_mnmajor_desc(base + static_cast<uint32_t>(kLaOffV), kLaTile * 128),
                   vdesc_few = sw128_mnmajor_desc(base + static_cast<uint32_t>(kLaOffV), kLaFew * 128);
    bool ok = true;
    int g = 0;
    for (int ic = 0; ok; ++ic) {
      LaItem w;
      if (!la_next_item(bars, ic, w, abort_flag)) { ok = false; break; }
      const int nt = __shfl_sync(0xffffffffu, w.nt, 0);
      if (nt < 0) break;
      for (int i = 0; i < nt && cr == 0; ++i, ++g) {  // the first CTA issues for both
        int kind, a, cnt;
        w.sp.tile(w.i0 + i, kind, a, cnt);
        const bool full = __shfl_sync(0xffffffffu, la_box_rows(cnt), 0) == kLaTile;
        if (!la_wait_all(&bars->v_full[0], g & 1, abort_flag)) { ok = false; break; }
        if (!la_wait_all(&bars->pfull, g & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t acc0 = i ? 1u : 0u;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          if (c == 1) {
            if (!la_wait_all(&bars->v_full[1], g & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
          }
          const uint32_t d = tmem + kLaColO + 128 * c;
          const uint64_t vd = vdesc + c * (kLaVGroup / 16), vf = vdesc_few + c * (kLaVGroup / 16);
          if (full) {
#pragma unroll
            for (int s = 0; s < 8; ++s)
              la_mma(d, pdesc + ((s >> 2) * kLaPanelBytes + 32 * (s & 3)) / 16, vd + 2048 * s / 16,
                     idesc_o, s ? 1u : acc0);
          } else {
#pragma unroll
            for (int s = 0; s < 2; ++s)
              la_mma(d, pdesc + 32 * s / 16, vf + 2048 * s / 16, idesc_o, s ? 1u : acc0);
          }
          la_commit_both(&bars->v_empty[c]);
        }
        if (!ok) break;
        la_commit_both(&bars->odone);
      }
    }
    if (cr == 0 && g > 0) {
      la_commit_both(&bars->drain[1], 1);
      if (lane == 0) mbar_wait_drain(&bars->drain[1], 0);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ value copies
    // (a warp of their own: their places become free at another pace than the keys')
    if (lane == 0) {
      const uint32_t v_full[2] = {la_map(&bars->v_full[0], 0), la_map(&bars->v_full[1], 0)};
      const uint32_t seen0 = la_map(&bars->v_seen, 0), seen1 = la_map(&bars->v_seen, 1);
      bool ok = true;
      int g = 0;
      for (int ic = 0; ok; ++ic) {
        const int slot = ic % kLaItems;
        if (!mbar_wait<false>(&bars->item_full[slot], (ic / kLaItems) & 1, abort_flag)) { ok = false; break; }
        const LaItem w = bars->item[slot];
        mbar_arrive(&bars->item_empty[slot]);
        if (w.nt < 0) break;
        for (int i = 0; i < w.nt && ok; ++i, ++g) {
          int kind, a, cnt;
          w.sp.tile(w.i0 + i, kind, a, cnt);
          const int box = la_box_rows(cnt);
          const int row = (kind ? w.rowd : w.row0) + a;
          for (int c = 0; c < 2; ++c) {
            // output MMA c has value columns 256 c .. : this CTA's 128 are panels 4 c + 2 cr and the next
            if (!mbar_wait<false>(&bars->v_empty[c], (g & 1) ^ 1, abort_flag)) { ok = false; break; }
            if (cr == 0) mbar_arrive_expect_tx(&bars->v_full[c], 2 * 2 * box * 128);
            la_load_3d(smem + kLaOffV + c * kLaVGroup, box == kLaTile ? &M.v : &M.v_few, v_full[c], row,
                       4 * c + 2 * cr);
          }
          if (cr == 0 && ok && !w.sp.whole(kind, a, cnt, P.n_sink)) {
            // both CTAs' softmax warps may read and clear these values; the other CTA's copies report to this one
            // (this warp waits for the values' MMAs anyway: the MMA warp's tiles took 1000 cycles longer with it)
            for (int c = 0; c < 2 && ok; ++c) {
              ok = mbar_wait<false>(&bars->v_full[c], g & 1, abort_flag);
              la_acquire(&bars->v_full[c], g & 1);
            }
            la_arrive_release(seen0);
            la_arrive_release(seen1);
          }
        }
      }
      if (!ok) la_settle();
    }
  }

  tc_fence_before();
  __syncthreads();
  la_cluster_sync();                                  // neither CTA ends while the other may read or signal it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Joins the parts of the items that cuts went through: blockIdx.x is the pair whose run the item begins in, its part
// 2 p + 1, the next pairs' parts 2 (p + 1), ...; blockIdx.y is one of its rows, four value columns a thread.  Parts
// whose lse is -inf are not read.
__global__ void __launch_bounds__(128)
    latent_attn_combine_kernel(const __grid_constant__ LatentAttnParams P) {
  __shared__ float s_lse[128];                        // at most 74 pairs
  const int p = blockIdx.x, r = blockIdx.y;
  const LaJoin join = P.joins[p];
  if (r >= join.nrows || join.parts <= 0) return;
  const auto at = [&](int k) { return static_cast<int64_t>(k == 0 ? 2 * p + 1 : 2 * (p + k)) * kLaRows + r; };
  const int parts = join.parts < 128 ? join.parts : 128;
  if (threadIdx.x < parts) s_lse[threadIdx.x] = __ldg(P.part_lse + at(threadIdx.x));
  __syncthreads();
  float m = neg_inf();
  for (int k = 0; k < parts; ++k) m = fmaxf(m, s_lse[k]);
  float den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < parts; ++k) {
    const float ls = s_lse[k];
    if (ls == neg_inf()) continue;
    const float w = expf(ls - m);
    const float4 v = __ldg(reinterpret_cast<const float4*>(P.part_o + at(k) * kAttnValue) + threadIdx.x);
    den += w;
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  const int64_t row = join.row0 + r;
  if (threadIdx.x == 0 && P.lse) P.lse[row] = den == 0.f ? neg_inf() : m + logf(den);
  const float4 o = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if (P.out_bf16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(o.x, o.y), c = __floats2bfloat162_rn(o.z, o.w);
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.out) + row * kAttnValue)[threadIdx.x] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&c));
  } else {
    reinterpret_cast<float4*>(static_cast<float*>(P.out) + row * kAttnValue)[threadIdx.x] = o;
  }
}

cudaError_t launch_latent_attn(const LaMaps& maps, const LatentAttnParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> attr_done{0};
  const cudaError_t e = smem_limit_once(attr_done, reinterpret_cast<const void*>(&latent_attn_kernel), kLaSmem);
  if (e != cudaSuccess) return e;
  latent_attn_kernel<<<static_cast<unsigned>(2 * p.pairs), kLaThreads, kLaSmem, st>>>(maps, p);
  return cudaGetLastError();
}

cudaError_t launch_latent_attn_combine(const LatentAttnParams& p, cudaStream_t st) {
  latent_attn_combine_kernel<<<dim3(static_cast<unsigned>(p.pairs), kLaRows), 128, 0, st>>>(p);
  return cudaGetLastError();
}

// How the work is laid out, from what the host knows: at most `items` items of at most `tiles` tiles.  Whole items in
// turn unless equal runs are shorter by more than 5 percent and the join's cost (about 4 tiles: a launch and the
// parts' way through memory).  An item's own cost counts two tiles in this choice (with kLaItemCost, 32 x 8 tokens x 16
// heads over a window of 512 rows would be cut, 28 us for 22, and 30 tokens x 128 heads, 27 for 20).  74 pairs run at
// once.
struct LaLayout {
  int pairs, cut;
};
inline LaLayout la_layout(int64_t items, int64_t tiles) {
  constexpr int64_t kPairs = 74, kOwn = 2;
  const int64_t weight = tiles + kOwn, total = items * weight;
  const int64_t whole = (items + kPairs - 1) / kPairs * weight;
  const int64_t runs = total < kPairs ? total : kPairs;
  const int64_t cut = (total + runs - 1) / runs + 4;
  const int64_t places = items * (tiles + kLaItemCost);
  LaLayout l;
  l.cut = 100 * whole > 105 * cut;
  l.pairs = static_cast<int>(l.cut ? (places < kPairs ? places : kPairs) : items < kPairs ? items : kPairs);
  return l;
}

}  // namespace lsi
