// Rotary positions of the queries and keys of a packed batch, forward and
// backward, with one to four position axes.
//
// Pair i of a head's first `rot` elements turns by theta = pos[axis(i), t] *
// freq_i; the backward pass turns by -theta (the rotation's transpose).  An
// angle matters only modulo one turn, so a frequency is held as the fraction
// freq_i / 2 pi of a turn a position, scaled by 2^64: the 64-bit product with
// the integer position wraps exactly at whole turns, and positions near 2^31
// lose nothing (the fraction's own error, 2^-65 turns, times the position).
// Sine and cosine then come from the top 32 bits of the product: reduced to
// [-1/8, 1/8] of a turn around the nearest quarter, evaluated by their Taylor
// series (truncation below 2e-9), and turned by the quarter.
//
// HBM-bound: each element is read once and written once.  A thread holds
// eight pairs of a token (16-byte vectors that neighbouring threads hold side by
// side) and walks several heads of it with the same sines and cosines in
// registers, its loads of all heads in flight before the angles are computed.
// 32768 tokens of 32 + 2 heads in bf16 take 90-100 us (571 MB, 87-97 % of the
// measured copy rate), an fp32 interleaved backward of 9973 tokens 55-57 us (93-96 %).
#include "sm100.cuh"

namespace infllm2 {

namespace rope {

constexpr int kThreads = 256;

__device__ __forceinline__ void sincos_turns(uint32_t f, float& s, float& c) {
  const uint32_t quarter = (f + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(f - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float x2 = x * x;
  // x - x^3/3! + x^5/5! - x^7/7! + x^9/9!  and  1 - x^2/2! + ... - x^10/10!
  const float ps = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), 0.f);
  const float sx = fmaf(x, ps, x);
  const float cx =
      fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f),
           1.f);
  s = (quarter & 1) ? cx : sx;
  c = (quarter & 1) ? sx : cx;
  if (quarter & 2) s = -s;
  if ((quarter + 1) & 2) c = -c;
}

// position x turns, modulo one turn, in units of 2^-32 turn
__device__ __forceinline__ uint32_t angle(int32_t pos, uint64_t turns) {
  return static_cast<uint32_t>((static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns) >> 32);
}

__device__ __forceinline__ void turn_pair(float& u, float& v, float c, float s) {
  const float x = u;
  u = x * c - v * s;
  v = v * c + x * s;
}

struct Args {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const int32_t* pos;   // [n_axes, total]
  int32_t total, h_q, h_kv, d, rot, n_axes, back;
  int32_t bound[3];     // first pair of axis 1, 2, 3
  uint64_t turns[INFLLM2_ROPE_MAX_PAIRS];
};

// 16 bytes of elements
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int W = 8;
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = r; }
};
template <>
struct Vec<float> {
  static constexpr int W = 4;
  float4 r;
  __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w; }
  __device__ __forceinline__ void set(const float (&x)[4]) { r = make_float4(x[0], x[1], x[2], x[3]); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = r; }
};

// A head has d / 2W couples of vectors, 8 / W of them a thread: couple p is the
// vectors at W p and rot/2 + W p (W pairs), or (INTER) those at W p and d/2 + W p (W/2
// pairs each); elements past rot are copied.  Needs rot % 16 == 0.  A thread walks
// heads hg, hg + HG, ... (HPT of them) of its token, query heads first, then key heads.
template <typename T, bool INTER, int HPT>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Args a, uint32_t HG, int nc_shift) {
  constexpr int W = Vec<T>::W, S = 8 / W;
  __shared__ uint64_t turns[INFLLM2_ROPE_MAX_PAIRS];
  const int c = threadIdx.x & ((1 << nc_shift) - 1);
  const uint32_t item = blockIdx.x * (kThreads >> nc_shift) + (threadIdx.x >> nc_shift);
  const uint32_t t = item / HG, hg = item - t * HG;
  const bool live = t < static_cast<uint32_t>(a.total);
  if (threadIdx.x < a.rot / 2) turns[threadIdx.x] = a.turns[threadIdx.x];
  const int half = a.rot >> 1;
  int e0[S], e1[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int p = c + (s << nc_shift), past = p - half / W;
    if (INTER) {
      e0[s] = W * p;
      e1[s] = (a.d >> 1) + W * p;
    } else {
      e0[s] = past < 0 ? W * p : a.rot + W * past;
      e1[s] = past < 0 ? half + W * p : a.rot + ((a.d - a.rot) >> 1) + W * past;
    }
  }

  Vec<T> x0[HPT][S], x1[HPT][S];
  int32_t ps[4] = {0, 0, 0, 0};
  const int heads = a.h_q + a.h_kv;
  if (live) {
    for (int ax = 0; ax < 4; ++ax)
      if (ax < a.n_axes) ps[ax] = __ldg(a.pos + static_cast<int64_t>(ax) * a.total + t);
#pragma unroll
    for (int j = 0; j < HPT; ++j) {
      const int h = hg + j * HG;
      if (h < heads) {
        const T* row = h < a.h_q ? static_cast<const T*>(a.q) + (static_cast<int64_t>(t) * a.h_q + h) * a.d
                                 : static_cast<const T*>(a.k) + (static_cast<int64_t>(t) * a.h_kv + (h - a.h_q)) * a.d;
#pragma unroll
        for (int s = 0; s < S; ++s) {
          x0[j][s].load(row + e0[s]);
          x1[j][s].load(row + e1[s]);
        }
      }
    }
  }
  __syncthreads();
  if (!live) return;
  float sn[S][W], cs[S][W];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < W; ++i) {
      // (past rot: no turn)
      const int pair = !INTER ? e0[s] + i : i < W / 2 ? e0[s] / 2 + i : e1[s] / 2 + i - W / 2;
      const int pos = pair >= a.bound[2] ? ps[3] : pair >= a.bound[1] ? ps[2] : pair >= a.bound[0] ? ps[1] : ps[0];
      sn[s][i] = 0.f;
      cs[s][i] = 1.f;
      if (pair < half) sincos_turns(angle(pos, turns[pair]), sn[s][i], cs[s][i]);
      if (a.back) sn[s][i] = -sn[s][i];
    }
#pragma unroll
  for (int j = 0; j < HPT; ++j) {
    const int h = hg + j * HG;
    if (h < heads) {
      T* row = h < a.h_q ? static_cast<T*>(a.q_out) + (static_cast<int64_t>(t) * a.h_q + h) * a.d
                         : static_cast<T*>(a.k_out) + (static_cast<int64_t>(t) * a.h_kv + (h - a.h_q)) * a.d;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float u[W], v[W];
        if (INTER) {
          if (e0[s] < a.rot) {
            x0[j][s].get(u);
#pragma unroll
            for (int i = 0; i < W; i += 2) turn_pair(u[i], u[i + 1], cs[s][i / 2], sn[s][i / 2]);
            x0[j][s].set(u);
          }
          if (e1[s] < a.rot) {
            x1[j][s].get(v);
#pragma unroll
            for (int i = 0; i < W; i += 2) turn_pair(v[i], v[i + 1], cs[s][(W + i) / 2], sn[s][(W + i) / 2]);
            x1[j][s].set(v);
          }
        } else if (e0[s] < half) {
          x0[j][s].get(u);
          x1[j][s].get(v);
#pragma unroll
          for (int i = 0; i < W; ++i) turn_pair(u[i], v[i], cs[s][i], sn[s][i]);
          x0[j][s].set(u);
          x1[j][s].set(v);
        }
        x0[j][s].store(row + e0[s]);
        x1[j][s].store(row + e1[s]);
      }
    }
  }
}

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(float& y, float x) { y = x; }

// Any even rot: a thread takes pair `threadIdx.x`, or copies an element past rot.  Only for a rot that the
// vectors above do not tile: its accesses are 2 or 4 bytes wide and its sines are computed again for each head, so
// 32768 tokens of 32 + 2 heads of 128 take 576 us in bf16 (rot 98 or 120; 90-92 us above with rot 96 or 128) and
// 573-579 us in fp32 (165-168 us); 16 tokens 2.0 us (3.1 us).
template <typename T>
__global__ void __launch_bounds__(128) rope_any_kernel(const __grid_constant__ Args a, int inter) {
  const int heads = a.h_q + a.h_kv, half = a.rot >> 1;
  const uint32_t t = blockIdx.x / heads, h = blockIdx.x - t * heads;
  const bool is_q = h < static_cast<uint32_t>(a.h_q);
  const int64_t off = is_q ? (static_cast<int64_t>(t) * a.h_q + h) * a.d
                           : (static_cast<int64_t>(t) * a.h_kv + (h - a.h_q)) * a.d;
  const T* x = static_cast<const T*>(is_q ? a.q : a.k) + off;
  T* y = static_cast<T*>(is_q ? a.q_out : a.k_out) + off;
  const int i = threadIdx.x;
  if (i < half) {
    const int ax = (i >= a.bound[0]) + (i >= a.bound[1]) + (i >= a.bound[2]);
    float s, c;
    sincos_turns(angle(__ldg(a.pos + static_cast<int64_t>(ax) * a.total + t), a.turns[i]), s, c);
    if (a.back) s = -s;
    const int e0 = inter ? 2 * i : i, e1 = inter ? 2 * i + 1 : half + i;
    const float u = to_f32(x[e0]), v = to_f32(x[e1]);
    from_f32(y[e0], u * c - v * s);
    from_f32(y[e1], v * c + u * s);
  }
  if (i >= a.rot && i < a.d) y[i] = x[i];
}

}  // namespace rope

template <typename T, bool INTER>
static cudaError_t launch_rope_typed(const rope::Args& a, cudaStream_t st) {
  const int nc = a.d / 16, nc_shift = a.d == 128 ? 3 : 2;
  const int64_t heads = static_cast<int64_t>(a.h_q) + a.h_kv;
  // several heads a thread (128 bytes each way) share the sines and cosines once
  // the grid still fills the GPU (a wave of 2048 threads an SM); below that, a head a thread
  constexpr int kMany = sizeof(T) == 2 ? 4 : 2;
  const bool many = static_cast<int64_t>(a.total) * heads * nc / kMany >= static_cast<int64_t>(num_sms()) * 2048;
  const int64_t HG = many ? (heads + kMany - 1) / kMany : heads;
  const int64_t items = static_cast<int64_t>(a.total) * HG;
  const int per = rope::kThreads / nc;
  const unsigned grid = static_cast<unsigned>((items + per - 1) / per);
  if (many)
    rope::rope_kernel<T, INTER, kMany><<<grid, rope::kThreads, 0, st>>>(a, static_cast<uint32_t>(HG), nc_shift);
  else
    rope::rope_kernel<T, INTER, 1><<<grid, rope::kThreads, 0, st>>>(a, static_cast<uint32_t>(HG), nc_shift);
  return cudaGetLastError();
}

cudaError_t launch_rope(const rope::Args& a, bool inter, bool f32, cudaStream_t st) {
  if (a.total == 0) return cudaSuccess;
  if (a.rot % 16 != 0) {   // pieces of eight pairs do not tile it
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.total) * (a.h_q + a.h_kv));
    if (f32) rope::rope_any_kernel<float><<<grid, 128, 0, st>>>(a, inter);
    else rope::rope_any_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(a, inter);
    return cudaGetLastError();
  }
  if (f32) return inter ? launch_rope_typed<float, true>(a, st) : launch_rope_typed<float, false>(a, st);
  return inter ? launch_rope_typed<__nv_bfloat16, true>(a, st) : launch_rope_typed<__nv_bfloat16, false>(a, st);
}

}  // namespace infllm2
