// The paged key-value cache: rows written into their pages (kept in bf16, or
// quantised to e4m3 with one fp32 scale a row) and read back as bf16.
//
// A row is the d values of one token and kv head.  8 bits: with a = max(max |x|,
// 2^-110), scale = a / 448 (e4m3's largest value) and y = e4m3(x * (448 / a)),
// each an fp32 operation rounded to nearest; 2^-110 keeps the scale of an
// all-zero row a normal number.  The maximum is taken over the bit patterns
// without the sign, in which infinities and NaN are the largest, so a row that
// holds one reads back as NaN instead of as finite values.
//
// HBM-bound.  A row belongs to d / 16 lanes, each with two 16-byte pieces of it
// (the row's K and V together: four independent loads a thread, on a write issued
// before the search for the row's sequence and page).  131072 8-bit rows of two kv
// heads are written in 34-37 us (floor 31.0 at the measured copy rate), 65521 read
// in 18.6 us (15.5), of which the launch is about 2.  Two rows a thread, for more
// loads behind one chain of lookups, were slower (37.0 and 19.1 us).
#include "sm100.cuh"

namespace infllm2 {

namespace paged {

constexpr int kThreads = 256;

struct Args {
  uint8_t* k_pages;
  uint8_t* v_pages;
  float* k_scale;
  float* v_scale;
  const int32_t* table;
  const int32_t* cu;      // [batch + 1]; null: one row a sequence
  const int32_t* start;   // [batch]; null: zeros
  int32_t n_pages, page_shift, batch, max_pages, h_kv;
  int32_t total;
};

// Row index (in rows of d values) of position `pos` of sequence b and kv head
// g, or -1 when the position or its page is out of range (recorded).
__device__ __forceinline__ int64_t page_row(const Args& a, int b, int64_t pos, int g) {
  if (pos >= static_cast<int64_t>(a.max_pages) << a.page_shift) {
    record_status(INFLLM2_ERR_DEVICE_BOUNDS);
    return -1;
  }
  const int32_t page = __ldg(a.table + static_cast<int64_t>(b) * a.max_pages + (pos >> a.page_shift));
  if (page < 0 || page >= a.n_pages) {
    record_status(INFLLM2_ERR_DEVICE_BOUNDS);
    return -1;
  }
  return ((static_cast<int64_t>(page) * a.h_kv + g) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

// Row index of packed token t and kv head g, or -1: rows outside every
// sequence and sequences with a negative start have none.
__device__ __forceinline__ int64_t packed_row(const Args& a, int t, int g) {
  int b = t, i = 0;
  if (a.cu) {
    b = find_sequence(a.cu, a.batch, t);
    i = t - __ldg(a.cu + b);
    if (i < 0 || t >= __ldg(a.cu + b + 1)) return -1;
  }
  const int s = a.start ? __ldg(a.start + b) : 0;
  if (s < 0) return -1;
  return page_row(a, b, static_cast<int64_t>(s) + i, g);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// two e4m3 values as two f16 (exact)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

__device__ __forceinline__ uint2 quantise8(const uint4& x, float r) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y[i] = e4m3x2(__uint_as_float(w[i] << 16) * r, __uint_as_float(w[i] & 0xffff0000u) * r);
  return make_uint2(y[0] | (y[1] << 16), y[2] | (y[3] << 16));
}

// e4m3 * scale (fp32), rounded to bf16
__device__ __forceinline__ uint4 dequantise8(const uint2& y, float s) {
  const uint32_t in[2] = {y.x, y.y};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = f16x2_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(in[i >> 1] >> (16 * (i & 1)))));
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x * s, f.y * s);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t absmax2(uint32_t m, const uint4& x) {
  m = __vmaxu2(m, x.x & 0x7fff7fffu);
  m = __vmaxu2(m, x.y & 0x7fff7fffu);
  m = __vmaxu2(m, x.z & 0x7fff7fffu);
  return __vmaxu2(m, x.w & 0x7fff7fffu);
}

constexpr uint32_t kFloorBits = (127 - 110) << 7;   // bf16 2^-110

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads) write_kernel(const Args a, const uint4* __restrict__ K,
                                                         const uint4* __restrict__ V) {
  constexpr int L = D / 16;               // lanes a row
  const uint32_t row = blockIdx.x * (kThreads / L) + threadIdx.x / L;
  const int c = threadIdx.x % L;
  const bool live = row < static_cast<uint32_t>(a.total) * static_cast<uint32_t>(a.h_kv);
  uint4 x[2][2] = {};
  int64_t at = -1;
  if (live) {
    const int64_t src = static_cast<int64_t>(row) * (2 * L) + c;
    x[0][0] = __ldg(K + src); x[0][1] = __ldg(K + src + L);
    x[1][0] = __ldg(V + src); x[1][1] = __ldg(V + src + L);
    const uint32_t t = row / a.h_kv;
    at = packed_row(a, static_cast<int>(t), static_cast<int>(row - t * a.h_kv));
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint8_t* pages = kv ? a.v_pages : a.k_pages;
    if (F8) {
      uint32_t m = absmax2(absmax2(kFloorBits, x[kv][0]), x[kv][1]);
      m = max(m & 0xffffu, m >> 16);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float top = __uint_as_float(m << 16);
      const float r = __fdiv_rn(448.f, top);
      if (at >= 0) {
        uint2* dst = reinterpret_cast<uint2*>(pages + at * D);
        dst[c] = quantise8(x[kv][0], r);
        dst[c + L] = quantise8(x[kv][1], r);
        if (c == 0) (kv ? a.v_scale : a.k_scale)[at] = __fdiv_rn(top, 448.f);
      }
    } else if (at >= 0) {
      uint4* dst = reinterpret_cast<uint4*>(pages + at * (2 * D));
      dst[c] = x[kv][0];
      dst[c + L] = x[kv][1];
    }
  }
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads) read_kernel(const Args a, uint4* __restrict__ K, uint4* __restrict__ V) {
  constexpr int L = D / 16;
  const uint32_t row = blockIdx.x * (kThreads / L) + threadIdx.x / L;
  const int c = threadIdx.x % L;
  if (row >= static_cast<uint32_t>(a.total) * static_cast<uint32_t>(a.h_kv)) return;
  const uint32_t t = row / a.h_kv;
  const int64_t at = packed_row(a, static_cast<int>(t), static_cast<int>(row - t * a.h_kv));
  if (at < 0) return;
  const int64_t dst = static_cast<int64_t>(row) * (2 * L) + c;
  uint4 x[2][2];
  if (F8) {
    uint2 y[2][2];
    float s[2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint2* src = reinterpret_cast<const uint2*>((kv ? a.v_pages : a.k_pages) + at * D);
      y[kv][0] = src[c];
      y[kv][1] = src[c + L];
      s[kv] = (kv ? a.v_scale : a.k_scale)[at];
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      x[kv][0] = dequantise8(y[kv][0], s[kv]);
      x[kv][1] = dequantise8(y[kv][1], s[kv]);
    }
  } else {
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint4* src = reinterpret_cast<const uint4*>((kv ? a.v_pages : a.k_pages) + at * (2 * D));
      x[kv][0] = src[c];
      x[kv][1] = src[c + L];
    }
  }
  K[dst] = x[0][0];
  K[dst + L] = x[0][1];
  V[dst] = x[1][0];
  V[dst + L] = x[1][1];
}

template <int D, bool F8>
static void launch(const Args& a, bool write, const void* K, const void* V, cudaStream_t st) {
  constexpr int per = kThreads / (D / 16);
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.total) * a.h_kv + per - 1) / per);
  if (write)
    write_kernel<D, F8><<<grid, kThreads, 0, st>>>(a, static_cast<const uint4*>(K), static_cast<const uint4*>(V));
  else
    read_kernel<D, F8><<<grid, kThreads, 0, st>>>(a, static_cast<uint4*>(const_cast<void*>(K)),
                                                  static_cast<uint4*>(const_cast<void*>(V)));
}

}  // namespace paged

cudaError_t launch_paged_rows(const paged::Args& a, bool write, int d, bool f8, const void* K, const void* V,
                              cudaStream_t st) {
  if (a.total == 0) return cudaSuccess;
  if (d == 128) f8 ? paged::launch<128, true>(a, write, K, V, st) : paged::launch<128, false>(a, write, K, V, st);
  else f8 ? paged::launch<64, true>(a, write, K, V, st) : paged::launch<64, false>(a, write, K, V, st);
  return cudaGetLastError();
}

}  // namespace infllm2
