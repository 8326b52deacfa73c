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
// the rows any of them sees, in tiles of 64, with the running maximum and sum
// of the softmax:
//
//  - tensor memory holds 512 columns, and an fp32 output of 512 value columns
//    would take all of them; a CTA therefore keeps half of the value columns
//    (256) and two CTAs work on the same 128 query rows, each computing the
//    logits;
//  - of the query's nine 64-element panels the four of this CTA's value half
//    live in tensor memory as the MMAs' A operand and five in shared memory
//    (80 KB); a tile's value panels stay until its output is accumulated
//    (three tiles of them, 96 KB); the other five have one place each (40 KB),
//    free for the next tile as soon as the logits passed them.  A copy takes
//    four panels at once (a 3-D box of 64 elements x rows x panels): with one
//    panel a copy the issue alone took 2000 of a tile's 3200 cycles.  The logits
//    take the value panels first, so both kinds of copies run about 1500
//    cycles ahead.  A value panel is staged once: the logits read it as
//    K-major keys and the output as MN-major values (the same bytes);
//  - the logits of tile i + 1 are issued before the output of tile i, so the
//    softmax of a tile runs beside the MMAs of the next;
//  - the weights go back to tensor memory as bf16 (A operand of the output);
//    the output is rescaled only when a row's maximum grew by more than 16
//    (in log2 units: weights stay below 2^16, which neither bf16 nor fp32
//    holds less exactly than weights below 1); the sinks, a few rows, come
//    after the window, so that the first reference is the maximum of many.
//
// Rounding to fewer bits: the weights (bf16, half a step is 2^-8 of a weight; the sum that
// divides the output is that of the rounded weights, so they still sum to 1)
// and the output when it is asked for in bf16.  Logits, sums, lse are fp32.
//
// Masked places weigh exactly 0 whatever they hold: a tile that not every row
// sees whole is checked for logits that are not finite at masked places, and
// only then the staged values are searched for elements that are not finite
// (a weight of 0 times one of them would be NaN) and cleared.  A visible row
// with a NaN or +inf logit makes its own query row NaN, and no other.
//
// Few query rows over a long span: the tiles are split over n_split CTA pairs,
// each writing its part (fp32, with its lse) to the workspace, and
// latent_attn_combine_kernel joins the parts.

#pragma once

#include "common.cuh"
#include "sparse_attn.cuh"

namespace lsi {

constexpr int kLaRows = 128;                          // query rows per CTA: the MMA's M
constexpr int kLaTile = 64;                           // cache rows per tile
constexpr int kLaPanelBytes = kLaTile * 128;          // 8 KB: 64 elements of 64 rows
constexpr int kLaVPanels = 4;                         // value panels of a CTA's half
constexpr int kLaTPanels = 5;                         // panels only the logits read
constexpr int kLaQTmem = 4;                           // query panels in tensor memory
constexpr int kLaQSmem = 5;                           // query panels in shared memory
constexpr int kLaQPanelBytes = kLaRows * 128;         // 16 KB
constexpr int kLaVBuf = kLaVPanels * kLaPanelBytes;  // 32 KB: the value panels of a tile
constexpr int kLaVBufs = 3;
constexpr int kLaTFirst = 4;                          // key-only panels freed by a commit of their own
constexpr int kLaThreads = 6 * 32;                    // copies, MMA, 4 softmax / epilogue warps
constexpr int kLaColO = 0, kLaColS = 256, kLaColQ = 384;            // tensor-memory columns
constexpr float kLaLazy = 16.f;                       // log2 growth of a maximum that forces a rescale
constexpr int kLaMaxSplit = 64;

struct LaBars {
  uint64_t qfull, qstage, qtmem;     // query: shared-memory panels landed; staged ones landed; in tensor memory
  uint64_t t_full;                   // a tile's key-only panels have landed (two arrivals)
  uint64_t t_empty[2];               // the first four, the last one are read
  uint64_t v_full[kLaVBufs], v_empty[kLaVBufs];
  uint64_t sfull[2];                 // logits in tensor memory
  uint64_t pfull[2];                 // weights in tensor memory
  uint64_t odone;                    // output MMAs of a tile are complete
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};
constexpr size_t kLaOffV = size_t(kLaQSmem) * kLaQPanelBytes;
constexpr size_t kLaOffT = kLaOffV + kLaVBufs * size_t(kLaVBuf);
constexpr size_t kLaOffBars = kLaOffT + kLaTPanels * size_t(kLaPanelBytes);
constexpr size_t kLaSmem = 1024 /*align slack*/ + kLaOffBars + 256;
static_assert(sizeof(LaBars) <= 256, "barrier block");
static_assert(kLaSmem <= 232448, "shared memory budget");
// the query panels on their way to tensor memory take the second and third value buffer
constexpr size_t kLaOffStage = kLaOffV + kLaVBuf;
static_assert(kLaQTmem * kLaQPanelBytes == 2 * kLaVBuf, "the staged query panels fit two value buffers");
// the output's rows on their way out, a 16-byte pad apart (lanes on different banks)
constexpr int kLaOutPitch16 = 256 * 2 + 16, kLaOutPitch32 = 256 * 4 + 16;
static_assert(kLaRows * kLaOutPitch32 <= kLaVBufs * kLaVBuf + kLaTPanels * kLaPanelBytes, "output rows fit the ring");

struct LatentAttnParams {
  const uint16_t* q = nullptr;        // [T * H][576]
  const int32_t* q_start = nullptr;   // [B + 1]
  const int32_t* kv_len = nullptr;    // [B]: window: rows with the tokens' own; tree: context rows
  const int64_t* row_off = nullptr;   // [B] or nullptr (0)
  const uint64_t* tree = nullptr;     // [T][words] or nullptr: the window form
  int words = 0;
  int B = 0, T = 0, H = 0;
  int max_tiles = 0;                  // 128-row tiles per sequence that the grid covers
  int64_t n_rows = 0;
  int window = 0, align = 1, n_sink = 0;   // window <= 0 (tree only): the whole context
  float scale = 0.f;
  int n_split = 1;
  int out_bf16 = 0;
  void* out = nullptr;                // [T * H][512]
  float* lse = nullptr;               // [T * H] or nullptr
  float* part_o = nullptr;            // [n_split][T * H][512]
  float* part_lse = nullptr;          // [n_split][T * H]
};

// First row of the window of the token at position p.
__host__ __device__ inline int la_window_lo(int p, int window, int align) {
  if (window <= 0) return 0;
  const int x = p - window + 1;
  return x <= 0 ? 0 : x - x % align;
}

__device__ __forceinline__ uint64_t la_low_mask(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// The rows that a tile of query rows can see, cut into tiles of 64.
struct LaSpan {
  int sink_len;          // rows [0, sink_len): sinks apart from the window
  int lo, hi;            // window / context rows
  int drafted;           // drafted rows behind the context
  int n0, n1, n2;        // tiles of each
  int lo_max, hi_min;    // rows [lo_max, hi_min) are in every query row's window
  __device__ __forceinline__ int tiles() const { return n0 + n1 + n2; }
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

// First of the four value panels of a CTA of value half vh, first of the four that it only reads as keys besides
// panel 8 (rotary): half 0 has the values of panels 0-3, half 1 those of panels 4-7.
__device__ __forceinline__ int la_v_panel(int vh) { return 4 * vh; }
__device__ __forceinline__ int la_t_panel(int vh) { return 4 - 4 * vh; }

// Box of 64 elements x rows x panels: x in elements of a panel, y the row, z the panel.
__device__ __forceinline__ void la_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(y), "r"(z)
      : "memory");
}

// Rows of a tile as they are staged: 64, or 16 for a tile of at most 16 (panels lie that many rows apart).
__device__ __forceinline__ int la_box_rows(int cnt) { return cnt <= 16 ? 16 : kLaTile; }

// Warp-uniform bounded wait in which every lane tests the barrier: when the
// phase is complete already, the common case of the MMA warp, it costs one
// test and a vote.
__device__ __forceinline__ bool la_wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait(bar, parity, abort_flag);
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

// Four MMAs along one 64-element panel (K = 16 each): one election, the
// descriptors stepped by 32 bytes.  A in shared memory (a_desc) ...
__device__ __forceinline__ void la_mma_panel(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// ... and A in tensor memory (8 columns a step), B stepped by b_step.
template <int B_STEP>
__device__ __forceinline__ void la_mma_tmem_x4(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "add.s64 b1, %2, %5;\n\tadd.s64 b2, %2, %6;\n\tadd.s64 b3, %2, %7;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "n"(B_STEP / 16), "n"(2 * B_STEP / 16),
      "n"(3 * B_STEP / 16)
      : "memory");
}

// Sets the masked places of 32 logits to -inf; whether one of them (among the
// places `there` that the MMAs wrote) was not finite.
__device__ __forceinline__ bool la_mask_row(uint32_t (&v)[32], uint32_t vis, uint32_t there) {
  const uint32_t hidden = there & ~vis;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (hidden & (1u << j)) bad |= (v[j] & 0x7f800000u) == 0x7f800000u;
    if (!(vis & (1u << j))) v[j] = 0xff800000u;
  }
  return bad;
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
// Masked places hold -inf and weigh 0 (a scale of 0 takes them out by the mask: 0 * -inf is NaN).
template <bool MASKED>
__device__ __forceinline__ void la_row_weights(const uint32_t (&va)[32], const uint32_t (&vb)[32], uint64_t vis,
                                               float sl2, float ref, uint32_t (&pw)[32], float& l, float& lt) {
  const uint32_t vlo = static_cast<uint32_t>(vis), vhi = static_cast<uint32_t>(vis >> 32);
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
    if (MASKED) {
      const uint32_t w = e < 16 ? vlo : vhi;
      if (!(w & (1u << ((2 * e) & 31)))) p0 = 0.f;
      if (!(w & (1u << ((2 * e + 1) & 31)))) p1 = 0.f;
    }
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

// Tensor maps over rows of 9 panels of 64 elements, boxes of 64 elements x rows x panels, 128-byte swizzle.
struct LaMaps {
  CUtensorMap q4, q1;       // q rows: 128 x 4 panels, 128 x 1
  CUtensorMap kv4, kv1;     // latent rows: 64 x 4, 64 x 1
  CUtensorMap few4, few1;   // latent rows: 16 x 4, 16 x 1
};

// grid: B * max_tiles * n_split * 2 CTAs, the value half innermost.
__global__ void __launch_bounds__(kLaThreads, 1)
    latent_attn_kernel(const __grid_constant__ LaMaps M, const __grid_constant__ LatentAttnParams P) {
  extern __shared__ uint8_t la_raw[];
  uint8_t* smem = smem_align1024(la_raw);
  LaBars* bars = reinterpret_cast<LaBars*>(smem + kLaOffBars);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // ------------------------------------------------------------ this CTA's work
  int64_t bid = blockIdx.x;
  const int vh = static_cast<int>(bid & 1);
  bid >>= 1;
  const int split = static_cast<int>(bid % P.n_split);
  bid /= P.n_split;
  const int qtile = static_cast<int>(bid % P.max_tiles);
  const int b = static_cast<int>(bid / P.max_tiles);
  const int H = P.H;
  const int t0 = __ldg(P.q_start + b), t1 = __ldg(P.q_start + b + 1);
  if (t0 < 0 || t1 < t0 || t1 > P.T) {                // not a prefix of the tokens: nothing of it is computed
    if (threadIdx.x == 0) atomicOr(&g_fault, FAULT_BAD_INDEX);
    return;
  }
  const int n = t1 - t0;
  const int64_t seq_rows = static_cast<int64_t>(n) * H;
  if (seq_rows > static_cast<int64_t>(P.max_tiles) * kLaRows && threadIdx.x == 0)
    atomicOr(&g_fault, FAULT_BAD_INDEX);              // more tokens than max_q: the rest is not computed
  const int64_t r0 = static_cast<int64_t>(qtile) * kLaRows;
  if (r0 >= seq_rows) return;
  const int nrows = static_cast<int>(seq_rows - r0 < kLaRows ? seq_rows - r0 : kLaRows);
  const int64_t grow0 = static_cast<int64_t>(t0) * H + r0;          // first row in q / out
  const int tok_first = static_cast<int>(r0 / H), tok_last = static_cast<int>((r0 + nrows - 1) / H);
  const bool is_tree = P.tree != nullptr;
  int kv = __ldg(P.kv_len + b);
  const int64_t off = P.row_off ? __ldg(P.row_off + b) : 0;
  const int own = is_tree ? n : 0;                    // drafted rows behind kv
  if ((kv < 0 || off < 0 || off > P.n_rows || kv + static_cast<int64_t>(own) > P.n_rows - off) && threadIdx.x == 0)
    atomicOr(&g_fault, FAULT_BAD_INDEX);              // rows outside the cache are not seen
  kv = kv < 0 ? 0 : kv > P.n_rows ? static_cast<int>(P.n_rows) : kv;
  int avail = 0;                                      // rows of the sequence that the cache holds
  if (off >= 0 && off < P.n_rows)
    avail = static_cast<int>(P.n_rows - off < kv + static_cast<int64_t>(own) ? P.n_rows - off : kv + own);
  LaSpan sp;
  if (is_tree) {
    const int ctx = kv < avail ? kv : avail;
    sp.drafted = avail - ctx;
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
  const int all = sp.tiles();
  const int per = (all + P.n_split - 1) / P.n_split;
  const int i0 = split * per < all ? split * per : all;
  const int i1 = i0 + per < all ? i0 + per : all;
  const int nt = i1 - i0;

  if (threadIdx.x == 0) {
    mbar_init(&bars->qfull, 1);
    mbar_init(&bars->qstage, 1);
    mbar_init(&bars->qtmem, 4);
    mbar_init(&bars->t_full, 2);
    mbar_init(&bars->t_empty[0], 1);
    mbar_init(&bars->t_empty[1], 1);
    for (int i = 0; i < kLaVBufs; ++i) {
      mbar_init(&bars->v_full[i], 1);
      mbar_init(&bars->v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->sfull[i], 1);
      mbar_init(&bars->pfull[i], 4);
    }
    mbar_init(&bars->odone, 1);
    mbar_init(&bars->drain, 1);
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&M.q4);
    tma_prefetch_desc(&M.q1);
    tma_prefetch_desc(&M.kv4);
    tma_prefetch_desc(&M.kv1);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    if (lane == 0 && nt > 0) {
      mbar_arrive_expect_tx(&bars->qstage, kLaQTmem * kLaQPanelBytes);
      la_load_3d(smem + kLaOffStage, &M.q4, &bars->qstage, static_cast<int>(grow0), la_v_panel(vh));
      mbar_arrive_expect_tx(&bars->qfull, kLaQSmem * kLaQPanelBytes);
      la_load_3d(smem, &M.q4, &bars->qfull, static_cast<int>(grow0), la_t_panel(vh));
      la_load_3d(smem + 4 * kLaQPanelBytes, &M.q1, &bars->qfull, static_cast<int>(grow0), 8);
      bool ok = true;
      int nT = 0, nV = 0;                             // arrivals on t_full, value buffers filled
      int vs = 0, vph = 1;                            // value buffer and the parity that says it is free
      for (int i = 0; i < nt && ok; ++i) {
        int kind, a, cnt;
        sp.tile(i0 + i, kind, a, cnt);
        const int row = static_cast<int>(off + a + (kind ? kv : 0));
        const int box = la_box_rows(cnt);
        const CUtensorMap* four = box == kLaTile ? &M.kv4 : &M.few4;
        const CUtensorMap* one = box == kLaTile ? &M.kv1 : &M.few1;
        for (int g = 0; g < 3 && ok; ++g) {
          const int what = g == 0 ? 2 : g - 1;        // 0, 1: key-only panels; 2: values
          if (what == 2) {
            if (i == 1) ok = mbar_wait(&bars->qtmem, 0, abort_flag);   // the staged query panels are read
            if (ok) ok = mbar_wait(&bars->v_empty[vs], vph, abort_flag);
            if (!ok) break;
            mbar_arrive_expect_tx(&bars->v_full[vs], 4 * box * 128);
            la_load_3d(smem + kLaOffV + vs * kLaVBuf, four, &bars->v_full[vs], row, la_v_panel(vh));
            ++nV;
            if (++vs == kLaVBufs) { vs = 0; vph ^= 1; }
          } else {
            ok = mbar_wait(&bars->t_empty[what], (i & 1) ^ 1, abort_flag);
            if (!ok) break;
            uint8_t* dst = smem + kLaOffT;
            mbar_arrive_expect_tx(&bars->t_full, (what ? 1 : 4) * box * 128);
            if (what == 0)
              la_load_3d(dst, four, &bars->t_full, row, la_t_panel(vh));
            else
              la_load_3d(dst + kLaTFirst * box * 128, one, &bars->t_full, row, 8);
            ++nT;
          }
        }
      }
      // no copy is in flight when the CTA ends (matters after an abort only; a tile whose second half was never
      // asked for cannot complete its phase, so its first half is given the second's arrival)
      mbar_wait_drain(&bars->qstage, 0);
      mbar_wait_drain(&bars->qfull, 0);
      if (nT & 1) mbar_arrive(&bars->t_full);
      if (nT > 0) mbar_wait_drain(&bars->t_full, ((nT - 1) >> 1) & 1);
      for (int k = nV > kLaVBufs ? nV - kLaVBufs : 0; k < nV; ++k)
        mbar_wait_drain(&bars->v_full[k % kLaVBufs], (k / kLaVBufs) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t base = smem_u32(smem);
    constexpr uint32_t idesc_o = idesc_bf16_f32(kLaRows, kLaVPanels * 64) | (1u << 16);   // B MN-major
    bool ok = nt > 0;
    if (ok) ok = warp_wait(&bars->qtmem, 0, abort_flag);
    if (ok) ok = warp_wait(&bars->qfull, 0, abort_flag);
    tc_fence_after();
    int n16_prev = 0;
    int vs = 0, vph = 0, vprev = 0;
    for (int i = 0; i <= nt && ok; ++i) {
      int n16 = 0;
      const int vcur = vs;
      if (i < nt) {
        const int st = i & 1;
        int kind, a, cnt;
        sp.tile(i0 + i, kind, a, cnt);
        n16 = (cnt + 15) >> 4;
        const uint32_t idesc_s = idesc_bf16_f32(kLaRows, 16 * n16);
        const uint32_t d = tmem + kLaColS + 64 * st;
        const uint32_t pitch = la_box_rows(cnt) * 128;   // bytes between panels
        if (!la_wait_all(&bars->v_full[vs], vph, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t vb = base + static_cast<uint32_t>(kLaOffV) + vs * kLaVBuf;
#pragma unroll
        for (int p = 0; p < kLaVPanels; ++p)
          la_mma_tmem_x4<32>(d, tmem + kLaColQ + 32 * p, sw128_kmajor_desc(vb + p * pitch), idesc_s,
                             p ? 1u : 0u);
        if (!la_wait_all(&bars->t_full, i & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int p = 0; p < kLaTPanels; ++p) {
          la_mma_panel(d, sw128_kmajor_desc(base + p * kLaQPanelBytes),
                       sw128_kmajor_desc(base + static_cast<uint32_t>(kLaOffT) + p * pitch), idesc_s, 1u);
          if (p == kLaTFirst - 1) umma_commit_warp(&bars->t_empty[0]);
        }
        umma_commit_warp(&bars->sfull[st]);
        umma_commit_warp(&bars->t_empty[1]);
        if (++vs == kLaVBufs) { vs = 0; vph ^= 1; }
      }
      if (i > 0) {                                    // the output of the tile before
        const int j = i - 1, st = j & 1;
        if (!la_wait_all(&bars->pfull[st], (j >> 1) & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t vb = base + static_cast<uint32_t>(kLaOffV) + vprev * kLaVBuf;
        const uint32_t a_tmem = tmem + kLaColS + 64 * st;
        const uint64_t bdesc = sw128_mnmajor_desc(vb, n16_prev == 1 ? 16 * 128 : kLaPanelBytes);
        if (n16_prev == 4) {
          la_mma_tmem_x4<2048>(tmem + kLaColO, a_tmem, bdesc, idesc_o, j ? 1u : 0u);
        } else {
          for (int s = 0; s < n16_prev; ++s)
            umma_f16_tmem_a_warp(tmem + kLaColO, a_tmem + 8 * s, bdesc + s * (2048 / 16), idesc_o, (j | s) ? 1u : 0u);
        }
        umma_commit_warp(&bars->v_empty[vprev]);
        umma_commit_warp(&bars->odone);
      }
      n16_prev = n16;
      vprev = vcur;
    }
    // all MMAs this warp started are complete once `drain` flips
    if (nt > 0) {
      umma_commit_warp(&bars->drain);
      if (lane == 0) mbar_wait_drain(&bars->drain, 0);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int quad = warp & 3;                        // warps 2-5: tensor-memory lanes 32 * (warp & 3) ..
    const int r = quad * 32 + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const bool live = r < nrows;
    const int tok = static_cast<int>((r0 + (live ? r : nrows - 1)) / H);
    bool ok = true;
    if (nt > 0) {
      // the staged query panels of this row into tensor memory
      ok = warp_wait(&bars->qstage, 0, abort_flag);
      for (int p = 0; p < kLaQTmem && ok; ++p) {
        uint32_t w[32];
        const uint8_t* src = smem + kLaOffStage + p * kLaQPanelBytes + r * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(src + ((c ^ (r & 7)) << 4));
          w[4 * c] = v.x;
          w[4 * c + 1] = v.y;
          w[4 * c + 2] = v.z;
          w[4 * c + 3] = v.w;
        }
        tmem_st_32x32(trow + kLaColQ + 32 * p, w);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->qtmem);
    }
    // this row's visible rows of the sequence: [0, hi) cut by the sinks and the window
    int hi, lo;
    const uint64_t* branch = nullptr;
    if (is_tree) {
      branch = P.tree + static_cast<int64_t>(t0 + tok) * P.words;
      int depth = 0;
      if (P.window > 0) {
        for (int w = 0; w < P.words; ++w) depth += __popcll(__ldg(branch + w) & la_low_mask(n - 64 * w));
        depth = depth > 0 ? depth - 1 : 0;
      }
      hi = sp.hi;
      lo = la_window_lo(kv + depth, P.window, P.align);
    } else {
      const int p = kv - n + tok;
      hi = p + 1 < avail ? p + 1 : avail;
      lo = la_window_lo(p, P.window, P.align);
    }
    // logits in log2 units; below 0 the logits' signs are turned instead
    const bool turn = P.scale < 0.f;
    const float sl2 = fabsf(P.scale) * 1.4426950408889634f;
    float m = neg_inf(), l = 0.f, lt = 0.f;           // reference, sum of the weights, of the rounded weights
    int vs = 0;
    for (int i = 0; i < nt && ok; ++i) {
      const int st = i & 1;
      int kind, a, cnt;
      sp.tile(i0 + i, kind, a, cnt);
      const bool whole = kind == 0 && cnt == kLaTile && a + kLaTile <= sp.hi_min &&
                         (a + kLaTile <= P.n_sink || a >= sp.lo_max);
      uint64_t vis = ~0ull;
      if (!whole) {
        if (kind == 0)
          vis = la_low_mask(hi - a < cnt ? hi - a : cnt) & (la_low_mask(P.n_sink - a) | ~la_low_mask(lo - a));
        else
          vis = __ldg(branch + (a >> 6)) & la_low_mask(cnt);
      }
      if (!warp_wait(&bars->sfull[st], (i >> 1) & 1, abort_flag)) { ok = false; break; }
      tc_fence_after();
      uint32_t va[32], vb[32];
      const uint32_t scol = trow + kLaColS + 64 * st;
      tmem_ld_32x32_nowait(scol, va);
      tmem_ld_32x32_nowait(scol + 32, vb);
      tmem_wait_ld(va);
      tmem_wait_ld(vb);
      if (turn) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          va[j] ^= 0x80000000u;
          vb[j] ^= 0x80000000u;
        }
      }
      if (!whole) {
        const uint64_t there = la_low_mask(16 * ((cnt + 15) >> 4));
        const bool bad = la_mask_row(va, static_cast<uint32_t>(vis), static_cast<uint32_t>(there)) |
                         la_mask_row(vb, static_cast<uint32_t>(vis >> 32), static_cast<uint32_t>(there >> 32));
        // A row that holds something not finite gives every query row a logit that is not finite, so each
        // warp finds out for its own query rows, and clears the staged values before its own arrival (two
        // warps that clear the same piece store the same bytes).
        if (__any_sync(0xffffffffu, bad)) {
          uint4* v4 = reinterpret_cast<uint4*>(smem + kLaOffV + vs * kLaVBuf);
          for (int e = lane; e < kLaVPanels * 8 * la_box_rows(cnt); e += 32) {
            uint4* at = v4 + e;
            uint4 x = *at;
            uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if ((xw[k] & 0x7f80u) == 0x7f80u) xw[k] &= 0xffff0000u;
              if ((xw[k] & 0x7f800000u) == 0x7f800000u) xw[k] &= 0x0000ffffu;
            }
            *at = x;
          }
          fence_proxy_async_smem();
        }
      }
      const float mt = la_row_max(va, vb, sl2);
      const bool grow = mt > m + kLaLazy;             // true at the first visible finite logit
      if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? (m == neg_inf() ? 0.f : la_exp2(m - mt)) : 1.f;
        if (grow) m = mt;
        l *= f;
        lt *= f;
        if (i > 0) {
          if (!warp_wait(&bars->odone, (i - 1) & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          for (int c = 0; c < 8; ++c) {
            uint32_t o[32];
            tmem_ld_32x32_nowait(trow + kLaColO + 32 * c, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st_32x32(trow + kLaColO + 32 * c, o);
          }
        }
      }
      const float ref = m == neg_inf() ? 0.f : m;
      uint32_t pw[32];
      if (whole)
        la_row_weights<false>(va, vb, vis, sl2, ref, pw, l, lt);
      else
        la_row_weights<true>(va, vb, vis, sl2, ref, pw, l, lt);
      tmem_st_32x32(scol, pw);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->pfull[st]);
      if (++vs == kLaVBufs) vs = 0;
    }
    // ------------------------------------------------------------ output
    // The logits of the last tile say that the output of tile nt - 3 is complete, so its phase and the next
    // one are waited for in turn (a wait for the last phase alone could meet the one two before it).
    if (ok && nt > 1) ok = warp_wait(&bars->odone, (nt - 2) & 1, abort_flag);
    if (ok && nt > 0) ok = warp_wait(&bars->odone, (nt - 1) & 1, abort_flag);
    if (ok) {
      tc_fence_after();
      const bool empty = l == 0.f;                    // nothing visible (or only -inf logits)
      const float inv = empty ? 0.f : 1.f / lt;
      const int64_t row = grow0 + r;
      const bool parts = P.n_split > 1;
      if (vh == 0 && live) {
        const float v = empty ? neg_inf() : (m + log2f(l)) * 0.6931471805599453f;
        if (parts)
          P.part_lse[static_cast<int64_t>(split) * P.T * H + row] = v;
        else if (P.lse)
          P.lse[row] = v;
      }
      // rows through shared memory (free now: every copy and MMA of the CTA is done), so that a store covers
      // a row's 512 bytes (one bulk copy per row took 3000 cycles to issue; this takes 600)
      const bool wide = parts || !P.out_bf16;
      uint8_t* stage = smem + kLaOffV + r * (wide ? kLaOutPitch32 : kLaOutPitch16);
      for (int c = 0; c < 8; ++c) {
        uint32_t o[32];
        if (nt > 0) {
          tmem_ld_32x32_nowait(trow + kLaColO + 32 * c, o);
          tmem_wait_ld(o);
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = empty ? 0u : __float_as_uint(__uint_as_float(o[k]) * inv);
        if (wide) {
          uint4* dst = reinterpret_cast<uint4*>(stage + 128 * c);
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(stage + 64 * c);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const __nv_bfloat162 h =
                  __floats2bfloat162_rn(__uint_as_float(o[8 * k + 2 * x]), __uint_as_float(o[8 * k + 2 * x + 1]));
              w[x] = *reinterpret_cast<const uint32_t*>(&h);
            }
            dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      __syncwarp();
      const uint32_t keep = __ballot_sync(0xffffffffu, live && !(parts && empty));   // an empty part is not read
      uint8_t* dst0 = parts ? reinterpret_cast<uint8_t*>(P.part_o + static_cast<int64_t>(split) * P.T * H * kAttnValue)
                            : static_cast<uint8_t*>(P.out);
      const int size = wide ? 4 : 2;
      const uint8_t* src0 = smem + kLaOffV + quad * 32 * (wide ? kLaOutPitch32 : kLaOutPitch16) + 16 * lane;
      dst0 += ((grow0 + quad * 32) * kAttnValue + 256 * vh) * size + 16 * lane;
#pragma unroll 8
      for (int rr = 0; rr < 32; ++rr) {               // a warp writes its rows one by one, 512 bytes an access
        if (!((keep >> rr) & 1u)) continue;
        if (wide) {
          const uint4 v = *reinterpret_cast<const uint4*>(src0 + rr * kLaOutPitch32);
          const uint4 w = *reinterpret_cast<const uint4*>(src0 + rr * kLaOutPitch32 + 512);
          *reinterpret_cast<uint4*>(dst0 + rr * (kAttnValue * 4)) = v;
          *reinterpret_cast<uint4*>(dst0 + rr * (kAttnValue * 4) + 512) = w;
        } else {
          *reinterpret_cast<uint4*>(dst0 + rr * (kAttnValue * 2)) =
              *reinterpret_cast<const uint4*>(src0 + rr * kLaOutPitch16);
        }
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the split form: a block of 128 threads per row, four
// value columns a thread; parts whose lse is -inf are not read.  Rows behind
// the last sequence are left as they were.
__global__ void __launch_bounds__(128)
    latent_attn_combine_kernel(const __grid_constant__ LatentAttnParams P) {
  const int64_t row = blockIdx.x;
  const int64_t rows = static_cast<int64_t>(P.T) * P.H;
  const int last = __ldg(P.q_start + P.B);
  if (row < static_cast<int64_t>(__ldg(P.q_start)) * P.H || row >= static_cast<int64_t>(last) * P.H) return;
  float m = neg_inf();
  for (int s = 0; s < P.n_split; ++s) m = fmaxf(m, __ldg(P.part_lse + s * rows + row));
  float den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < P.n_split; ++s) {
    const float ls = __ldg(P.part_lse + s * rows + row);
    if (ls == neg_inf()) continue;
    const float w = expf(ls - m);
    const float4 v = __ldg(reinterpret_cast<const float4*>(P.part_o + (s * rows + row) * kAttnValue) + threadIdx.x);
    den += w;
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
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
  const int64_t blocks = static_cast<int64_t>(p.B) * p.max_tiles * p.n_split * 2;
  latent_attn_kernel<<<static_cast<unsigned>(blocks), kLaThreads, kLaSmem, st>>>(maps, p);
  return cudaGetLastError();
}

cudaError_t launch_latent_attn_combine(const LatentAttnParams& p, cudaStream_t st) {
  latent_attn_combine_kernel<<<static_cast<unsigned>(static_cast<int64_t>(p.T) * p.H), 128, 0, st>>>(p);
  return cudaGetLastError();
}

// Number of CTA pairs that share one tile of query rows.  `pairs` pairs cover
// the query rows, each over at most `tiles` tiles of the cache; the machine
// runs 74 pairs at once.  A tile costs about 1 us, a pair about 6 tiles more
// for its query, its first copies and its output, and the combine about 4
// (with the launch): the split that makes the longest chain shortest.
inline int la_splits(int64_t pairs, int64_t tiles) {
  int best = 1;
  int64_t best_cost = 0;
  const int64_t most = tiles < kLaMaxSplit ? tiles : kLaMaxSplit;
  for (int64_t s = 1; s <= (most > 1 ? most : 1); ++s) {
    const int64_t waves = (pairs * s + 73) / 74;
    const int64_t cost = waves * ((tiles + s - 1) / s + 6) + (s > 1 ? 4 : 0);
    if (s == 1 || cost < best_cost) {
      best = static_cast<int>(s);
      best_cost = cost;
    }
  }
  return best;
}

}  // namespace lsi
