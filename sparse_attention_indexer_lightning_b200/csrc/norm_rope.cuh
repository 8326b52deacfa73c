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
//   fp8: scale = max |y| / 448 (1 for a row of zeros), code = e4m3(y / scale)
//
// Bound by bytes: every element is read and written once.  A warp takes one
// row at a time, 8 elements (16 bytes) of it per lane and step, held in
// registers as fp32 between the two passes that a norm needs; only the
// rotation's partners cross lanes, through the warp's own strip of shared
// memory.  The angle is formed in 64 bits (at a position of ten million an
// fp32 product is off by a radian) and reduced to half turns before the fp32
// sine and cosine; a block works on the heads of one token, so that an angle
// is computed once per block and not per head.

#pragma once

#include "common.cuh"

namespace lsi {

constexpr int kNrMaxDim = 1024;
constexpr int kNrWarps = 8;
constexpr int kNrMaxRope = 256;
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

__device__ __forceinline__ float nr_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float nr_warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// STEPS = ceil(d / 256): 16-byte pieces per lane.
template <int STEPS>
__global__ void __launch_bounds__(kNrWarps * 32)
    norm_rope_kernel(const __grid_constant__ NormRopeParams P) {
  __shared__ float s_cos[kNrMaxRope / 2], s_sin[kNrMaxRope / 2];
  __shared__ float s_mid[kNrWarps][kNrMaxRope];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x / P.blocks_per_token;
  const int h0 = (blockIdx.x - t * P.blocks_per_token) * P.chunk;
  const int half = P.rope / 2;
  {
    const int64_t pos = half > 0 ? __ldg(P.pos + t) : 0;
    for (int i = threadIdx.x; i < half; i += kNrWarps * 32) {
      // the angle in half turns, reduced to [-1, 1]
      const double half_turns = static_cast<double>(pos) * static_cast<double>(__ldg(P.inv_freq + i)) * 0.31830988618379067;
      const double r = half_turns - 2.0 * rint(0.5 * half_turns);
      sincospif(static_cast<float>(r), &s_sin[i], &s_cos[i]);
    }
  }
  __syncthreads();
  const int pieces = P.d >> 3;
  const int heads = P.part[0].heads + P.part[1].heads;
  const int h_end = h0 + P.chunk < heads ? h0 + P.chunk : heads;
  for (int hh = h0 + warp; hh < h_end; hh += kNrWarps) {
    const bool second = hh >= P.part[0].heads;
    const NormRows& R = P.part[second ? 1 : 0];
    const int h = second ? hh - P.part[0].heads : hh;
    int64_t orow = t;
    if (R.slots) {
      orow = __ldg(R.slots + t);
      if (orow < 0 || orow >= R.out_rows) {           // -1: the token has no row
        if (orow != -1 && lane == 0) atomicOr(&g_fault, FAULT_BAD_INDEX);
        continue;
      }
    }
    const uint4* src = reinterpret_cast<const uint4*>(R.x + t * R.x_stride + static_cast<int64_t>(h) * P.d);
    float x[STEPS][8];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int c = 32 * s + lane;
      const uint4 v = c < pieces ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[s][2 * k] = __uint_as_float(w[k] << 16);
        x[s][2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
    if (R.norm != NORM_NONE) {                        // norm_dim is a multiple of 8: whole pieces
      const int np = P.norm_dim >> 3;
      const float inv_n = 1.f / static_cast<float>(P.norm_dim);
      float mu = 0.f;
      if (R.norm == NORM_LAYER) {
        float a = 0.f;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
          if (32 * s + lane < np) {
#pragma unroll
            for (int k = 0; k < 8; ++k) a += x[s][k];
          }
        mu = nr_warp_sum(a) * inv_n;
      }
      float q = 0.f;
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
        if (32 * s + lane < np) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[s][k] -= mu;
            q = fmaf(x[s][k], x[s][k], q);
          }
        }
      const float rs = 1.f / sqrtf(nr_warp_sum(q) * inv_n + P.eps);
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int c = 32 * s + lane;
        if (c < np) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float y = x[s][k] * rs;
            if (R.weight) y *= __ldg(R.weight + 8 * c + k);
            if (R.bias) y += __ldg(R.bias + 8 * c + k);
            x[s][k] = y;
          }
        }
      }
    }
    if (half > 0) {
      // the rotated part through the warp's strip, so that any pairing and any offset is a plain read
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int c = 32 * s + lane;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int i = 8 * c + k - P.rope_off;
          if (c < pieces && i >= 0 && i < P.rope) s_mid[warp][i] = x[s][k];
        }
      }
      __syncwarp();
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int c = 32 * s + lane;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int i = 8 * c + k - P.rope_off;
          if (c < pieces && i >= 0 && i < P.rope) {
            const bool hi = P.interleaved ? (i & 1) : (i >= half);
            const int pair = P.interleaved ? (i >> 1) : (hi ? i - half : i);
            const float other = s_mid[warp][P.interleaved ? (i ^ 1) : (hi ? i - half : i + half)];
            const float co = s_cos[pair], si = s_sin[pair];
            x[s][k] = hi ? fmaf(x[s][k], co, other * si) : fmaf(x[s][k], co, -(other * si));
          }
        }
      }
      __syncwarp();
    }
    const int64_t at = orow * R.heads + h;
    if (P.fp8) {
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[s][k]));
      top = nr_warp_max(top);
      const float sc = top > 0.f ? top / 448.f : 1.f;
      if (lane == 0) R.scale[at] = sc;
      uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(R.out) + at * P.d);
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int c = 32 * s + lane;
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint16_t two;                               // d.hi = e4m3(a), d.lo = e4m3(b)
          asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
              : "=h"(two)
              : "f"(x[s][2 * k + 1] / sc), "f"(x[s][2 * k] / sc));
          w[k >> 1] |= static_cast<uint32_t>(two) << (16 * (k & 1));
        }
        if (c < pieces) dst[c] = make_uint2(w[0], w[1]);
      }
    } else {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(R.out) + at * P.d);
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int c = 32 * s + lane;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(x[s][2 * k], x[s][2 * k + 1]);
          w[k] = *reinterpret_cast<const uint32_t*>(&b);
        }
        if (c < pieces) dst[c] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

cudaError_t launch_norm_rope(const NormRopeParams& p0, int num_sms, cudaStream_t st) {
  NormRopeParams p = p0;
  const int heads = p.part[0].heads + p.part[1].heads;
  if (p.T == 0 || heads == 0) return cudaSuccess;
  // a block takes all heads of a token unless the tokens alone would leave SMs without a block
  int split = 1;
  while (static_cast<int64_t>(p.T) * split < num_sms && split * kNrWarps < heads) split *= 2;
  p.chunk = (heads + split - 1) / split;
  p.blocks_per_token = (heads + p.chunk - 1) / p.chunk;
  const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(p.T) * p.blocks_per_token);
  const int threads = kNrWarps * 32;
  switch ((p.d + 255) / 256) {
    case 1: norm_rope_kernel<1><<<blocks, threads, 0, st>>>(p); break;
    case 2: norm_rope_kernel<2><<<blocks, threads, 0, st>>>(p); break;
    case 3: norm_rope_kernel<3><<<blocks, threads, 0, st>>>(p); break;
    default: norm_rope_kernel<4><<<blocks, threads, 0, st>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace lsi
