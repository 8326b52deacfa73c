// Norm of the query heads and of the key, the position rotation, and the write
// to bf16 rows or to fp8 codes with a scale (the 132-byte key of the fp8
// indexer, "03 long context", section "The Architectural Answer: Read Less of
// the Past"), in one pass over each row.
//
// For a head row x of d elements, of which the first norm_dim are normed and
// the `rope` elements from rope_off on are rotated:
//
//   y[i] = (x[i] - mu) * rsqrt(mean((x - mu)^2) + eps) * w[i] + b[i]    i < norm_dim
//          (mu = 0 for the root-mean-square norm; y = x without a norm)
//   (a, b) -> (a cos f - b sin f, b cos f + a sin f),  f = pos * inv_freq[i]
//          for the pairs (2i, 2i + 1), interleaved, or (i, i + rope / 2)
//   fp8: scale = max |y| / 448 (1 for a row of zeros, else 2^-149 at least), code = e4m3(y / scale)
//
// Long rows are bound by bytes: every element is read and written once; short
// ones by the wait for a batch of rows and the instructions that follow.  LPR
// lanes (8, 16 or 32, whichever leaves the fewest idle) share a row, each
// holding STEPS pieces of 8 elements in fp32 between the passes that a norm
// needs.  A block works on heads of one token: its angles are formed once (in
// 64 bits: at a position of ten million an fp32 product is off by a radian;
// reduced to half turns before the fp32 sine and cosine), and a lane keeps
// those of its pieces in registers for all its rows.  Where the rotated part is
// whole pieces of one step (ALIGNED), a rotation's partners are in the same
// piece (interleaved) or in the same registers of another lane, one shuffle
// away; any other offset goes through a strip of shared memory.
//
// Measured on a B200: 2048 x 129 rows of 576 elements 111 us, 5.5 TB/s (0.84 of
// the measured copy); 4096 x 33 rows of 128 elements to fp8 22 us (2.5 TB/s:
// 14 M warp instructions, the issue slots half used: neither bytes nor issue
// slots bound it, a warp loads its rows and works on them in turn).

#pragma once

#include "common.cuh"

namespace lsi {

constexpr int kNrMaxDim = 1024;
constexpr int kNrMaxRope = 256;
// Warps of a block: one for rows of one step (no warp waits while another forms the angles: 4096 x 33 rows of 128
// elements took 21 us, 26 with two warps, 33 with four), four for longer rows (2048 x 129 rows of 576 elements: 111 us,
// 117 with two).
constexpr int nr_warps(int steps) { return steps == 1 ? 1 : 4; }
constexpr float kNrTinyScale = 0x1p-126f;   // the smallest normal number: reciprocals of scales from here on are finite
enum : int { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };

struct NormRows {
  const uint16_t* x = nullptr;       // [T][heads][d], a token's rows x_stride elements apart
  int64_t x_stride = 0;
  int heads = 0;
  int norm = NORM_NONE;
  const float* weight = nullptr;     // [norm_dim] or nullptr (ones)
  const float* bias = nullptr;       // [norm_dim] or nullptr (zeros)
  void* out = nullptr;               // [rows][heads][d] bf16 or e4m3 codes
  float* scale = nullptr;            // [rows][heads], fp8 only
  const int64_t* slots = nullptr;    // [T] output row of token t (-1: none), or nullptr (row t)
  int64_t out_rows = 0;              // rows of out, with slots
};

struct NormRopeParams {
  NormRows part[2];                  // queries, keys (heads == 0: none)
  const int64_t* pos = nullptr;      // [T]
  const float* inv_freq = nullptr;   // [rope / 2]
  int T = 0, d = 0, norm_dim = 0, rope = 0, rope_off = 0, interleaved = 0, fp8 = 0;
  float eps = 0.f;
  int chunk = 1;                     // head rows per block
  int blocks_per_token = 1;
};

template <int LPR>
__device__ __forceinline__ float nr_row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LPR>
__device__ __forceinline__ float nr_row_max(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Elements c .. c + 7 of a vector, or `without` where there is none.
__device__ __forceinline__ void nr_load8(float (&w)[8], const float* __restrict__ p, int c, float without) {
  if (p == nullptr) {
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = without;
  } else if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {   // (the same for every piece of a vector)
    const float4 a = __ldg(reinterpret_cast<const float4*>(p + c)), b = __ldg(reinterpret_cast<const float4*>(p + c) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = __ldg(p + c + k);
  }
}

// One row (LPR lanes of the warp; the others work on other rows): norm, rotation, store.
// `on`: the row exists and is written; every lane takes part in the shuffles.
template <int LPR, int STEPS, bool ALIGNED>
__device__ __forceinline__ void nr_row(const NormRopeParams& P, const NormRows& R, float (&x)[STEPS][8], int lane_in,
                                       int64_t at, bool on, const float (&wr)[8], const float (&br)[8],
                                       const float (&rc)[8], const float (&rsn)[8], int rope_step, float* strip,
                                       const float* s_cos, const float* s_sin) {
  const int pieces = P.d >> 3;
  const int np = P.norm_dim >> 3;                     // norm_dim is a multiple of 8: whole pieces
  const int half = P.rope >> 1;
  if (R.norm != NORM_NONE) {                          // (the same for all rows of an operand)
    const float inv_n = 1.f / static_cast<float>(P.norm_dim);
    if (R.norm == NORM_LAYER) {
      float a = 0.f;
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
        if (LPR * s + lane_in < np) {
#pragma unroll
          for (int k = 0; k < 8; ++k) a += x[s][k];
        }
      const float mu = nr_row_sum<LPR>(a) * inv_n;
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
        if (LPR * s + lane_in < np) {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[s][k] -= mu;
        }
    }
    float q = 0.f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
      if (LPR * s + lane_in < np) {
#pragma unroll
        for (int k = 0; k < 8; ++k) q = fmaf(x[s][k], x[s][k], q);
      }
    const float rs = rsqrtf(nr_row_sum<LPR>(q) * inv_n + P.eps);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int c = LPR * s + lane_in;
      if (c < np) {
        if (STEPS == 1) {                             // the lane's weights are in registers
#pragma unroll
          for (int k = 0; k < 8; ++k) x[s][k] = fmaf(x[s][k] * rs, wr[k], br[k]);
        } else {
          float w[8];
          nr_load8(w, R.weight, 8 * c, 1.f);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[s][k] *= rs * w[k];
          if (R.bias) {
            nr_load8(w, R.bias, 8 * c, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[s][k] += w[k];
          }
        }
      }
    }
  }
  if (ALIGNED) {
    // the step that holds the rotated part; the pieces outside it stay as they are (an infinity too)
    if (half > 0) {
      const int j = LPR * rope_step + lane_in - (P.rope_off >> 3);   // piece of the rotated part
      const bool rotated = j >= 0 && 8 * j < P.rope;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        if (s != rope_step) continue;
        if (P.interleaved) {
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            const float a = x[s][k], b = x[s][k + 1];
            if (rotated) {
              x[s][k] = fmaf(a, rc[k], b * rsn[k]);
              x[s][k + 1] = fmaf(b, rc[k + 1], a * rsn[k + 1]);
            }
          }
        } else {
          const int hp = half >> 3;
          const bool second = j >= hp;
          const int partner = !rotated ? lane_in : second ? lane_in - hp : lane_in + hp;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float other = __shfl_sync(0xffffffffu, x[s][k], partner, LPR);
            if (rotated) x[s][k] = fmaf(x[s][k], rc[k], other * rsn[k]);
          }
        }
      }
    }
  } else {
    // through the row's strip, so that any pairing and any offset is a plain read
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int c = LPR * s + lane_in;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = 8 * c + k - P.rope_off;
        if (c < pieces && i >= 0 && i < P.rope) strip[i] = x[s][k];
      }
    }
    __syncwarp();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int c = LPR * s + lane_in;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = 8 * c + k - P.rope_off;
        if (c < pieces && i >= 0 && i < P.rope) {
          const bool second = P.interleaved ? (i & 1) : (i >= half);
          const int pair = P.interleaved ? (i >> 1) : (second ? i - half : i);
          const float other = strip[P.interleaved ? (i ^ 1) : (second ? i - half : i + half)];
          const float co = s_cos[pair], si = s_sin[pair];
          x[s][k] = second ? fmaf(x[s][k], co, other * si) : fmaf(x[s][k], co, -(other * si));
        }
      }
    }
    __syncwarp();
  }
  if (P.fp8) {
    float top = 0.f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[s][k]));
    top = nr_row_max<LPR>(top);
    // Products with 1 / 448 and 1 / scale for the quotients: an ulp or two of fp32, far below an e4m3 step.  The
    // reciprocal of a scale below kNrTinyScale may leave fp32 (and a zero's code would be 0 * inf): such a row's quotients
    // are formed of 2^64 times both.
    const float sc = top > 0.f ? fmaxf(top * (1.f / 448.f), 0x1p-149f) : 1.f;
    const float up = sc < kNrTinyScale ? 0x1p64f : 1.f;
    const float inv = __frcp_rn(sc * up);
    // (a warp's vote: a division in a branch of each lane's own took 34 us for 4096 x 33 rows of 128 elements, this 22)
    if (__any_sync(0xffffffffu, sc < kNrTinyScale)) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[s][k] *= up;
    }
    if (on && lane_in == 0) R.scale[at] = sc;
    uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(R.out) + at * P.d);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int c = LPR * s + lane_in;
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint16_t two;                                 // high byte: the first operand
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
            : "=h"(two)
            : "f"(x[s][2 * k + 1] * inv), "f"(x[s][2 * k] * inv));
        w[k >> 1] |= static_cast<uint32_t>(two) << (16 * (k & 1));
      }
      if (on && c < pieces) dst[c] = make_uint2(w[0], w[1]);
    }
  } else {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(R.out) + at * P.d);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int c = LPR * s + lane_in;
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[s][2 * k], x[s][2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&b);
      }
      if (on && c < pieces) dst[c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Heads h0 .. h1 of one operand of token t, by the block's warps from warp `w0` on.
template <int LPR, int STEPS, bool ALIGNED>
struct NrRows {
  static constexpr int kWarps = nr_warps(STEPS);
  static constexpr int kRows = 32 / LPR;              // rows a warp works on at once
  static constexpr int kDeep = STEPS == 1 ? 2 : 1;    // and one after another, their loads issued together
  static constexpr int kStride = kWarps * kRows;
  uint4 raw[kDeep][STEPS];

  __device__ __forceinline__ void fetch(const NormRopeParams& P, const NormRows& R, const uint16_t* xt, int base,
                                        int h1, int lane_in) {
    const int pieces = P.d >> 3;
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int h = base + u * kStride;
      const uint4* src = reinterpret_cast<const uint4*>(xt + h * P.d);
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int c = LPR * s + lane_in;
        raw[u][s] = h < h1 && c < pieces ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  __device__ __forceinline__ void run(const NormRopeParams& P, const NormRows& R, int t, int h0, int h1, int w0,
                                      bool fetched, int warp, int lane, const float (&rc)[8], const float (&rsn)[8],
                                      int rope_step, float* strip, const float* s_cos, const float* s_sin) {
    const int lane_in = lane % LPR, sub = lane / LPR;
    const uint16_t* xt = R.x + t * R.x_stride;
    int64_t orow = t;
    bool has = true;
    if (R.slots) {
      orow = __ldg(R.slots + t);
      has = orow >= 0 && orow < R.out_rows;           // -1: the token has no row
      if (!has) {
        if (orow != -1 && threadIdx.x == 0 && h0 == 0) atomicOr(&g_fault, FAULT_BAD_INDEX);
        return;
      }
    }
    float wr[8], br[8];
    if (STEPS == 1) {
      const bool in = R.norm != NORM_NONE && lane_in < (P.norm_dim >> 3);
      nr_load8(wr, in ? R.weight : nullptr, 8 * lane_in, 1.f);
      nr_load8(br, in ? R.bias : nullptr, 8 * lane_in, 0.f);
    }
    const int64_t at0 = orow * R.heads;
    const int first = h0 + ((warp + kWarps - w0) % kWarps) * kRows;
    for (int base = first; base < h1; base += kDeep * kStride) {
      if (!fetched || base != first) fetch(P, R, xt, base + sub, h1, lane_in);
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        if (base + u * kStride >= h1) break;          // (uniform over the warp)
        const int h = base + sub + u * kStride;
        const bool on = h < h1;
        float x[STEPS][8];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const uint32_t w[4] = {raw[u][s].x, raw[u][s].y, raw[u][s].z, raw[u][s].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[s][2 * k] = __uint_as_float(w[k] << 16);
            x[s][2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
          }
        }
        nr_row<LPR, STEPS, ALIGNED>(P, R, x, lane_in, at0 + (on ? h : 0), on, wr, br, rc, rsn, rope_step, strip, s_cos,
                                    s_sin);
      }
    }
  }
};

template <int LPR, int STEPS, bool ALIGNED>
__global__ void __launch_bounds__(nr_warps(STEPS) * 32)
    norm_rope_kernel(const __grid_constant__ NormRopeParams P) {
  using Rows = NrRows<LPR, STEPS, ALIGNED>;
  __shared__ float s_cos[kNrMaxRope / 2], s_sin[kNrMaxRope / 2];
  __shared__ float s_strip[ALIGNED ? 1 : Rows::kWarps * Rows::kRows][ALIGNED ? 1 : kNrMaxRope];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lane_in = lane % LPR, sub = lane / LPR;
  const int t = blockIdx.x / P.blocks_per_token;
  // the block's share of the token's rows, the queries' first
  const int r0 = (blockIdx.x - t * P.blocks_per_token) * P.chunk, nq = P.part[0].heads;
  const int r1 = r0 + P.chunk < nq + P.part[1].heads ? r0 + P.chunk : nq + P.part[1].heads;
  const int q0 = r0 < nq ? r0 : nq, q1 = r1 < nq ? r1 : nq;
  const int k0 = r0 > nq ? r0 - nq : 0, k1 = r1 > nq ? r1 - nq : 0;
  const int half = P.rope >> 1;

  Rows rows;
  const bool early = q0 < q1;                         // the first queries' loads are in flight while the angles are formed
  if (early)
    rows.fetch(P, P.part[0], P.part[0].x + t * P.part[0].x_stride, q0 + warp * Rows::kRows + sub, q1, lane_in);
  if (half > 0) {
    const int64_t pos = __ldg(P.pos + t);
    for (int i = threadIdx.x; i < half; i += Rows::kWarps * 32) {
      // the angle in half turns, reduced to [-1, 1]
      const double half_turns =
          static_cast<double>(pos) * static_cast<double>(__ldg(P.inv_freq + i)) * 0.31830988618379067;
      const double r = half_turns - 2.0 * rint(0.5 * half_turns);
      sincospif(static_cast<float>(r), &s_sin[i], &s_cos[i]);
    }
  }
  __syncthreads();
  // the cosines and the signed sines of this lane's piece of the rotated step (ALIGNED)
  float rc[8], rsn[8];
  const int rope_step = ALIGNED ? (P.rope_off >> 3) / LPR : 0;
  if (ALIGNED) {
    const int j = LPR * rope_step + lane_in - (P.rope_off >> 3);
    const bool in = j >= 0 && 8 * j < P.rope;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int e = 8 * j + k;                        // element of the rotated part; the first of a pair subtracts
      const bool second = P.interleaved ? (k & 1) : e >= half;
      const int pair = P.interleaved ? e >> 1 : second ? e - half : e;
      rc[k] = in ? s_cos[pair] : 1.f;
      rsn[k] = in ? (second ? s_sin[pair] : -s_sin[pair]) : 0.f;
    }
  }
  float* strip = s_strip[ALIGNED ? 0 : warp * Rows::kRows + sub];
  if (early)
    rows.run(P, P.part[0], t, q0, q1, 0, true, warp, lane, rc, rsn, rope_step, strip, s_cos, s_sin);
  if (k0 < k1)                                        // the keys start at the warp that has the fewest queries
    rows.run(P, P.part[1], t, k0, k1, ((q1 - q0 + Rows::kRows - 1) / Rows::kRows) % Rows::kWarps, false, warp, lane, rc, rsn,
             rope_step, strip, s_cos, s_sin);
}

template <int LPR, int STEPS>
inline void nr_launch(const NormRopeParams& p, unsigned blocks, cudaStream_t st) {
  // the rotated part is whole pieces of one step (interleaved pairs lie inside a piece anyway)
  const int piece = p.rope_off >> 3, last = (p.rope_off + p.rope - 1) >> 3;
  const bool aligned = p.rope == 0 || (p.rope_off % 8 == 0 && p.rope % (p.interleaved ? 8 : 16) == 0 &&
                                       piece / LPR == last / LPR);
  if (aligned)
    norm_rope_kernel<LPR, STEPS, true><<<blocks, nr_warps(STEPS) * 32, 0, st>>>(p);
  else
    norm_rope_kernel<LPR, STEPS, false><<<blocks, nr_warps(STEPS) * 32, 0, st>>>(p);
}

cudaError_t launch_norm_rope(const NormRopeParams& p0, int num_sms, cudaStream_t st) {
  NormRopeParams p = p0;
  const int heads = p.part[0].heads + p.part[1].heads;
  if (p.T == 0 || heads == 0) return cudaSuccess;
  const int pieces = p.d / 8;
  // A block takes all heads of a token unless that leaves SMs short of blocks: of 16 one-warp blocks each (500 tokens x
  // 33 rows of 128 elements: 6.3 us, 11.9 undivided), of two larger ones.
  const bool one_step = pieces <= 16 || (pieces > 24 && pieces <= 32);
  const int64_t want = static_cast<int64_t>(one_step ? 16 : 2) * num_sms;
  int split = 1;
  while (static_cast<int64_t>(p.T) * split < want && 4 * split < heads) split *= 2;
  p.chunk = (heads + split - 1) / split;
  p.blocks_per_token = (heads + p.chunk - 1) / p.chunk;
  const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(p.T) * p.blocks_per_token);
  // lanes per row and pieces per lane: the fewest idle lanes for d / 8 pieces
  if (pieces <= 8) nr_launch<8, 1>(p, blocks, st);
  else if (pieces <= 16) nr_launch<16, 1>(p, blocks, st);
  else if (pieces <= 24) nr_launch<8, 3>(p, blocks, st);
  else if (pieces <= 32) nr_launch<32, 1>(p, blocks, st);
  else if (pieces <= 64) nr_launch<32, 2>(p, blocks, st);
  else if (pieces <= 72) nr_launch<8, 9>(p, blocks, st);
  else nr_launch<32, 4>(p, blocks, st);
  return cudaGetLastError();
}

}  // namespace lsi
