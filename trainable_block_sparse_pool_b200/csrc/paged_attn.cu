// Attention of one new token a sequence over its whole paged key-value cache:
// the dense side of the dense/sparse switch at decode (the sparse side is
// decode.cu).
//
// For query head h of kv group g and the first n = len[b] positions u,
//   z_u = scale log2(e) q_h . k_u,  lse = log2 sum_u 2^z_u,  out = sum_u 2^(z_u - lse) v_u,
// in one pass with a running maximum and sum.  Every key and value is read once
// for the group's G <= 16 query heads, so the kernel is bound by HBM; 4 d G
// flop a (token, kv head) go to warp-level mma.sync m16n8k16, whose 16 rows are
// the group's heads.
//
// Split.  Lengths are known on the device only, so the grid is fixed (one CTA
// an SM, kWarps warps) and every warp works alone: the 16-token units of all
// (sequence, kv head) pairs, in order, are cut into equal ranges, one a warp,
// whatever the lengths.  A piece of a pair that begins and ends within one
// range is written out by its warp; the others leave a normalised partial and
// its log-sum-exp in the workspace, and a second kernel (programmatic dependent
// launch) joins them in ascending order.  Nothing waits on another CTA.
//
// A warp streams tiles of 8 KB (K and V of 16, 32 or 64 tokens) through its own
// kStages-deep cp.async ring.  Rows past the piece are filled with zeros, not
// read, so what lies in unwritten slots never enters a product.
//
// 8 bits.  K and V go from e4m3 to f16 exactly.  q is scaled to f16 by a power
// of two a head (its 8 significant bits are kept down to 2^-29 of the head's
// largest element, and 2^-39 of it absolutely).  A value's scale multiplies its
// probability: w_u = p_u * scale_u / R * 2^15 in f16, with R a power of two no
// less than any scale seen, so w keeps 11 bits where p_u scale_u >= 2^-29 R.
#include "sm100.cuh"

namespace infllm2 {

namespace pattn {

using dec::QFrag;
using dec::cp_async_commit;
using dec::cp_async_wait_n;
using dec::ldsm_x4_t;
using dec::load_qfrag;
using dec::mma16816;

constexpr int kWarps = 8;
constexpr int kStages = 3;
constexpr int kUnit = 16;           // tokens; every page size is a multiple of it
constexpr int kHalf = 4096;         // bytes of K, and of V, in a stage

__device__ __forceinline__ void mma16816_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// `bytes` (0 .. 16) from src, zeros after them
__device__ __forceinline__ void cp_async16_part(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

struct Args {
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  const int32_t* len;
  const __nv_bfloat16* q;
  void* out;
  float* lse;             // [batch, h_q] or null
  int64_t* prefix;        // workspace: [batch + 1] units of the sequences before b (one kv head)
  float* part_o;          // workspace: [2 * workers][G][D]
  float* part_lse;        // workspace: [2 * workers][G]
  int32_t n_pages, page_shift, batch, max_pages, h_kv, G, ctas, out_f32;
  float scale_log2;
};

// units of a sequence; a length outside [0, capacity] counts as 0 (recorded by CTA 0)
__device__ __forceinline__ int seq_units(const Args& a, int b) {
  const int n = __ldg(a.len + b);
  const bool ok = n >= 0 && n <= static_cast<int64_t>(a.max_pages) << a.page_shift;
  if (!ok && blockIdx.x == 0) record_status(INFLLM2_ERR_DEVICE_BOUNDS);
  return ok ? (n + kUnit - 1) / kUnit : 0;
}

// range of worker w of nw over `total` units
__device__ __forceinline__ int64_t range_begin(int64_t total, int w, int nw) { return total * w / nw; }

template <int D, bool F8>
struct Cfg {
  static constexpr int kRow = F8 ? D : 2 * D;         // bytes a row
  static constexpr int kTile = kHalf / kRow;          // tokens a tile
  static constexpr int CH = kRow / 16;                // 16-byte pieces a row
  static constexpr int kScale = F8 ? 8 * kTile : 0;   // bytes of scales in a stage
  static constexpr int kStage = 2 * kHalf + kScale;
  static constexpr int kSmem = kWarps * kStages * kStage;
  static constexpr int NT = kTile / 8;                // 8-key tiles of S
  static constexpr int OT = D / 8;                    // 8-column tiles of O
};

// Shared-memory byte of 16-byte piece c of tile row r.  Rows of 128 bytes or
// more keep their own lines with the piece XORed by the row; two 64-byte rows
// share a line, XORed by the line.
template <int CH>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  if (CH >= 8) return r * (CH * 16) + ((c ^ (r & 7)) << 4);
  return (r >> 1) * 128 + (((r & 1) * 4 + (c ^ ((r >> 1) & 3))) << 4);
}

// Key n of an 8-key tile of S is the tile's token key_token(n).  The order is
// free (probabilities and values use the same one); this one lets the eight
// lanes of each shared-memory phase, two keys of four pieces or four values of
// two, meet all eight 16-byte banks groups.
template <int CH>
__device__ __forceinline__ int key_token(int n) {
  const int t = n >> 1, e = n & 1;
  if (CH >= 8) return (2 * t + (t >> 1)) ^ (4 * e);
  return ((t & 1) | ((t & 2) << 1)) ^ (3 * e);
}

// Walks the tiles of a warp's range.
struct Walk {
  int b, g, n, u, ue;   // sequence, kv head, its units, next unit, end of this piece
  int64_t left;         // units of the range after this piece
  int tok_end;          // tokens of the piece end here
};

__device__ __forceinline__ void walk_piece(const Args& a, Walk& w) {
  const int64_t take = min(static_cast<int64_t>(w.n - w.u), w.left);
  w.ue = w.u + static_cast<int>(take);
  w.left -= take;
  w.tok_end = min(__ldg(a.len + w.b), w.ue * kUnit);
}

// to the next tile; false when the range is done
template <int kTile>
__device__ __forceinline__ bool walk_next(const Args& a, Walk& w) {
  w.u += kTile / kUnit;
  if (w.u < w.ue) return true;
  if (w.left <= 0) return false;
  if (++w.g == a.h_kv) {
    w.g = 0;
    do { ++w.b; w.n = seq_units(a, w.b); } while (w.n == 0);
  }
  w.u = 0;
  walk_piece(a, w);
  return true;
}

template <int D, bool F8>
__device__ __forceinline__ void issue_tile(const Args& a, const Walk& w, uint32_t stage, int lane) {
  using C = Cfg<D, F8>;
  constexpr int RPI = 32 / C::CH;   // rows an instruction
  const int tok0 = w.u * kUnit;
  const int nv = min(C::kTile, w.tok_end - tok0);
  const int32_t* row = a.table + static_cast<int64_t>(w.b) * a.max_pages;
  const int r0 = lane / C::CH, c = lane % C::CH;
  const int mask = (1 << a.page_shift) - 1;
  int64_t base[C::kTile / kUnit];   // first row of each 16-token group (-1: nothing to read)
#pragma unroll
  for (int i = 0; i < C::kTile / kUnit; ++i) {
    const int tok = tok0 + i * kUnit;
    base[i] = -1;
    if (i * kUnit < nv) {
      const int page = __ldg(row + (tok >> a.page_shift));
      if (page >= 0 && page < a.n_pages)
        base[i] = ((static_cast<int64_t>(page) * a.h_kv + w.g) << a.page_shift) + (tok & mask);
      else
        record_status(INFLLM2_ERR_DEVICE_BOUNDS);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * RPI + r0;
    const int64_t at = base[i * RPI / kUnit];
    const bool ok = r < nv && at >= 0;
    const int64_t off = ok ? (at + (r & (kUnit - 1))) * C::kRow + c * 16 : 0;
    const uint32_t dst = stage + piece_at<C::CH>(r, c);
    cp_async16_part(dst, a.k_pages + off, ok ? 16 : 0);
    cp_async16_part(dst + kHalf, a.v_pages + off, ok ? 16 : 0);
  }
  if (F8) {
    // scales: pieces of four tokens, K's then V's
    constexpr int P = C::kTile / 4;
    if (lane < 2 * P) {
      const int t = 4 * (lane % P);
      int64_t at = -1;
#pragma unroll
      for (int i = 0; i < C::kTile / kUnit; ++i)
        if (t / kUnit == i) at = base[i];
      const int bytes = at >= 0 ? max(0, min(16, 4 * (nv - t))) : 0;
      const float* src = lane < P ? a.k_scale : a.v_scale;
      cp_async16_part(stage + 2 * kHalf + lane * 16, bytes > 0 ? src + at + (t & (kUnit - 1)) : src, bytes);
    }
  }
}

// Query heads as A fragments: bf16 as they are, or (F8) f16 scaled to
// [2^14, 2^15) by a power of two a head; `unscale` undoes it.
template <int D, bool F8>
struct Query {
  uint32_t a[D / 16][4];
  float unscale[2];
};

template <int D, bool F8>
__device__ __forceinline__ void load_query(Query<D, F8>& f, const __nv_bfloat16* q, int lane, int G) {
  const int gid = lane >> 2, tig = lane & 3;
  if (!F8) {
    QFrag<D> t;
    load_qfrag<D>(t, q, lane, G);
#pragma unroll
    for (int p = 0; p < D / 32; ++p) {
      f.a[2 * p][0] = t.lo[p].x; f.a[2 * p][1] = t.hi[p].x; f.a[2 * p][2] = t.lo[p].y; f.a[2 * p][3] = t.hi[p].y;
      f.a[2 * p + 1][0] = t.lo[p].z; f.a[2 * p + 1][1] = t.hi[p].z;
      f.a[2 * p + 1][2] = t.lo[p].w; f.a[2 * p + 1][3] = t.hi[p].w;
    }
    f.unscale[0] = f.unscale[1] = 1.f;
    return;
  }
  // k step 4j + i covers d = 16 (tig + 4j) + 4i + {0, 1} and + {2, 3} in this thread
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int h = gid + 8 * s;
    uint4 v[D / 32];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const uint4* p = reinterpret_cast<const uint4*>(q + h * D + 16 * (tig + 4 * j));
      v[2 * j] = h < G ? p[0] : make_uint4(0, 0, 0, 0);
      v[2 * j + 1] = h < G ? p[1] : make_uint4(0, 0, 0, 0);
      top = paged::absmax2(paged::absmax2(top, v[2 * j]), v[2 * j + 1]);
    }
    top = max(top & 0xffffu, top >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // bf16 exponent e: |q| < 2^(e - 126); scale by 2^(141 - e)
    const int e = min(max(static_cast<int>(top >> 7), 15), 254);
    const float up = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
    f.unscale[s] = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4& x = v[2 * j + (i >> 1)];
        const uint32_t w0 = (i & 1) ? x.z : x.x, w1 = (i & 1) ? x.w : x.y;
        f.a[4 * j + i][s] = pack_f16(__uint_as_float(w0 << 16) * up, __uint_as_float(w0 & 0xffff0000u) * up);
        f.a[4 * j + i][2 + s] = pack_f16(__uint_as_float(w1 << 16) * up, __uint_as_float(w1 & 0xffff0000u) * up);
      }
  }
}

template <int D, bool F8>
struct State {
  float o[D / 8][4];
  float m[2], l[2];   // running maximum (all four lanes of a head) and this lane's sum, heads gid and gid + 8
  int e_r;            // F8: R = 2^(e_r - 127)
};

template <int D, bool F8>
__device__ __forceinline__ void state_clear(State<D, F8>& s) {
#pragma unroll
  for (int i = 0; i < D / 8; ++i) s.o[i][0] = s.o[i][1] = s.o[i][2] = s.o[i][3] = 0.f;
  s.m[0] = s.m[1] = -INFINITY;
  s.l[0] = s.l[1] = 0.f;
  s.e_r = 16;
}

template <int D, bool F8>
__device__ __forceinline__ void attend_tile(State<D, F8>& st, const Query<D, F8>& q, uint32_t stage, int nv,
                                            float scale_log2, int lane) {
  using C = Cfg<D, F8>;
  const int gid = lane >> 2, tig = lane & 3;
  float z[C::NT][4];
  // S = Q K^T
#pragma unroll
  for (int t = 0; t < C::NT; ++t) {
    z[t][0] = z[t][1] = z[t][2] = z[t][3] = 0.f;
    const int r = 8 * t + key_token<C::CH>(gid);
#pragma unroll
    for (int j = 0; j < C::CH / 4; ++j) {
      const uint4 k = lds128(stage + piece_at<C::CH>(r, tig + 4 * j));
      if (F8) {
        const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mma16816_f16(z[t], q.a[4 * j + i], paged::e4m3x2_to_f16x2(static_cast<uint16_t>(w[i])),
                       paged::e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> 16)));
      } else {
        mma16816(z[t], q.a[2 * j], k.x, k.y);
        mma16816(z[t], q.a[2 * j + 1], k.z, k.w);
      }
    }
  }
  // scale and mask; the tile's maxima
  const int n0 = key_token<C::CH>(2 * tig), n1 = key_token<C::CH>(2 * tig + 1);
  const float s0 = scale_log2 * q.unscale[0], s1 = scale_log2 * q.unscale[1];
  float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int t = 0; t < C::NT; ++t) {
    float f0 = 1.f, f1 = 1.f;
    if (F8) {
      f0 = lds32(stage + 2 * kHalf + 4 * (8 * t + n0));
      f1 = lds32(stage + 2 * kHalf + 4 * (8 * t + n1));
    }
    const bool in0 = 8 * t + n0 < nv, in1 = 8 * t + n1 < nv;
    z[t][0] = in0 ? z[t][0] * (s0 * f0) : -INFINITY;
    z[t][1] = in1 ? z[t][1] * (s0 * f1) : -INFINITY;
    z[t][2] = in0 ? z[t][2] * (s1 * f0) : -INFINITY;
    z[t][3] = in1 ? z[t][3] * (s1 * f1) : -INFINITY;
    top[0] = fmaxf(top[0], fmaxf(z[t][0], z[t][1]));
    top[1] = fmaxf(top[1], fmaxf(z[t][2], z[t][3]));
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    top[s] = fmaxf(top[s], __shfl_xor_sync(0xffffffffu, top[s], 1));
    top[s] = fmaxf(top[s], __shfl_xor_sync(0xffffffffu, top[s], 2));
  }
  float back = 1.f;   // F8: R before / R now
  if constexpr (F8) {
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < C::kTile / 32; ++i)
      bits = max(bits, __float_as_uint(lds32(stage + 2 * kHalf + 4 * C::kTile + 4 * (lane + 32 * i))) & 0x7fffffffu);
    bits = __reduce_max_sync(0xffffffffu, bits);
    const int e = min(max(static_cast<int>((bits + 0x7fffffu) >> 23), 16), 250);
    if (e > st.e_r) {
      back = e - st.e_r > 126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + st.e_r - e) << 23);
      st.e_r = e;
    }
  }
  if (__any_sync(0xffffffffu, top[0] > st.m[0] || top[1] > st.m[1] || back != 1.f)) {
    float f[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const float m = fmaxf(st.m[s], top[s]);
      f[s] = st.m[s] == m ? 1.f : ex2(st.m[s] - m);   // equal infinities: nothing summed yet, or NaN below
      st.m[s] = m;
      st.l[s] *= f[s];
      f[s] *= back;
    }
#pragma unroll
    for (int i = 0; i < C::OT; ++i) {
      st.o[i][0] *= f[0]; st.o[i][1] *= f[0];
      st.o[i][2] *= f[1]; st.o[i][3] *= f[1];
    }
  }
  const float m0 = st.m[0] == -INFINITY ? 0.f : st.m[0], m1 = st.m[1] == -INFINITY ? 0.f : st.m[1];
  const float up = F8 ? __uint_as_float(static_cast<uint32_t>(254 + 15 - st.e_r) << 23) : 1.f;
  // probabilities as A fragments: P in bf16 (relative error 2^-9, that of the
  // output's own rounding), or w in f16; their sums stay in fp32 unrounded
  uint32_t p[C::NT / 2][4];
#pragma unroll
  for (int t = 0; t < C::NT; ++t) {
    float p0 = ex2(z[t][0] - m0), p1 = ex2(z[t][1] - m0), p2 = ex2(z[t][2] - m1), p3 = ex2(z[t][3] - m1);
    st.l[0] += p0 + p1;
    st.l[1] += p2 + p3;
    if (F8) {
      const float f0 = lds32(stage + 2 * kHalf + 4 * (C::kTile + 8 * t + n0)) * up;
      const float f1 = lds32(stage + 2 * kHalf + 4 * (C::kTile + 8 * t + n1)) * up;
      p[t >> 1][2 * (t & 1)] = pack_f16(p0 * f0, p1 * f1);
      p[t >> 1][2 * (t & 1) + 1] = pack_f16(p2 * f0, p3 * f1);
    } else {
      p[t >> 1][2 * (t & 1)] = pack_bf16(p0, p1);
      p[t >> 1][2 * (t & 1) + 1] = pack_bf16(p2, p3);
    }
  }
  // O += P V
  const uint32_t vs = stage + kHalf;
#pragma unroll
  for (int k = 0; k < C::NT / 2; ++k) {
    if (F8) {
      // a byte of four value rows: column d = 16 gid + i (8 gid + i for d = 64) of O's tile i
      const int r0 = 16 * k + n0, r1 = 16 * k + n1;
      constexpr int W = D / 32;   // words a row and lane
      uint32_t w[4][W];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (i & 1 ? r1 : r0) + (i >> 1) * 8;
        if (W == 4) {
          const uint4 v = lds128(vs + piece_at<C::CH>(r, gid));
          w[i][0] = v.x; w[i][1] = v.y; w[i][W - 2] = v.z; w[i][W - 1] = v.w;
        } else {
          const uint2 v = lds64(vs + piece_at<C::CH>(r, gid >> 1) + (gid & 1) * 8);
          w[i][0] = v.x; w[i][1] = v.y;
        }
      }
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint32_t lo0 = __byte_perm(w[0][j], w[1][j], 0x5140), lo1 = __byte_perm(w[0][j], w[1][j], 0x7362);
        const uint32_t hi0 = __byte_perm(w[2][j], w[3][j], 0x5140), hi1 = __byte_perm(w[2][j], w[3][j], 0x7362);
        mma16816_f16(st.o[4 * j], p[k], paged::e4m3x2_to_f16x2(static_cast<uint16_t>(lo0)),
                     paged::e4m3x2_to_f16x2(static_cast<uint16_t>(hi0)));
        mma16816_f16(st.o[4 * j + 1], p[k], paged::e4m3x2_to_f16x2(static_cast<uint16_t>(lo0 >> 16)),
                     paged::e4m3x2_to_f16x2(static_cast<uint16_t>(hi0 >> 16)));
        mma16816_f16(st.o[4 * j + 2], p[k], paged::e4m3x2_to_f16x2(static_cast<uint16_t>(lo1)),
                     paged::e4m3x2_to_f16x2(static_cast<uint16_t>(hi1)));
        mma16816_f16(st.o[4 * j + 3], p[k], paged::e4m3x2_to_f16x2(static_cast<uint16_t>(lo1 >> 16)),
                     paged::e4m3x2_to_f16x2(static_cast<uint16_t>(hi1 >> 16)));
      }
    } else {
      // four 8x8 matrices: keys 0-7 and 8-15 of the step, two 8-column tiles
      const int i = lane >> 3;
      const int r = 16 * k + (i & 1) * 8 + key_token<C::CH>(lane & 7);
#pragma unroll
      for (int j = 0; j < C::OT / 2; ++j) {
        uint32_t v[4];
        ldsm_x4_t(v, vs + piece_at<C::CH>(r, 2 * j + (i >> 1)));
        mma16816(st.o[2 * j], p[k], v[0], v[1]);
        mma16816(st.o[2 * j + 1], p[k], v[2], v[3]);
      }
    }
  }
}

// The G heads' normalised rows and log-sum-exps: to out and lse (slot < 0), or to partial `slot`.
template <int D, bool F8>
__device__ __forceinline__ void write_piece(const Args& a, State<D, F8>& st, int b, int g, int slot, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float l = st.l[s];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const int h = gid + 8 * s;
    if (h >= a.G) continue;
    // l = 0: every score was -inf; the row is empty
    float inv = l == 0.f ? 0.f : 1.f / l;
    if (F8) inv *= __uint_as_float(static_cast<uint32_t>(st.e_r - 15) << 23);
    const float lse = l == 0.f ? -INFINITY : st.m[s] + log2f(l);
    const int64_t row = (static_cast<int64_t>(b) * a.h_kv + g) * a.G + h;
    float* po = nullptr;
    if (slot >= 0) {
      po = a.part_o + (static_cast<int64_t>(slot) * a.G + h) * D;
      if (tig == 0) a.part_lse[static_cast<int64_t>(slot) * a.G + h] = lse;
    } else {
      if (a.out_f32) po = static_cast<float*>(a.out) + row * D;
      if (a.lse && tig == 0) a.lse[row] = lse;
    }
    __nv_bfloat16* pb = static_cast<__nv_bfloat16*>(a.out) + row * D;
    if (F8) {
      // this lane: columns [D/4 tig, D/4 (tig + 1)), tiles' first columns, then their second ones
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < D / 8; i += 4) {
          const float v0 = st.o[i][2 * s + e] * inv, v1 = st.o[i + 1][2 * s + e] * inv;
          const float v2 = st.o[i + 2][2 * s + e] * inv, v3 = st.o[i + 3][2 * s + e] * inv;
          const int d = D / 4 * tig + D / 8 * e + i;
          if (po) *reinterpret_cast<float4*>(po + d) = make_float4(v0, v1, v2, v3);
          else *reinterpret_cast<uint2*>(pb + d) = make_uint2(pack_bf16(v0, v1), pack_bf16(v2, v3));
        }
    } else {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float v0 = st.o[i][2 * s] * inv, v1 = st.o[i][2 * s + 1] * inv;
        const int d = 8 * i + 2 * tig;
        if (po) *reinterpret_cast<float2*>(po + d) = make_float2(v0, v1);
        else *reinterpret_cast<uint32_t*>(pb + d) = pack_bf16(v0, v1);
      }
    }
  }
}

template <int D, bool F8>
__global__ void __launch_bounds__(32 * kWarps, 1) attend_kernel(const __grid_constant__ Args a) {
  using C = Cfg<D, F8>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t chunk[32 * kWarps + 1];   // units (one kv head) before each thread's share of the sequences
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  dec::griddep_launch_dependents();

  // units of all sequences
  const int per = (a.batch + 32 * kWarps - 1) / (32 * kWarps);
  const int b_lo = min(a.batch, static_cast<int>(threadIdx.x) * per), b_hi = min(a.batch, b_lo + per);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += seq_units(a, b);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) chunk[warp] = incl;
  __syncthreads();
  int64_t before = 0;
  for (int w = 0; w < warp; ++w) before += chunk[w];
  __syncthreads();
  chunk[threadIdx.x + 1] = before + incl;
  if (threadIdx.x == 0) chunk[0] = 0;
  __syncthreads();
  const int64_t units = chunk[32 * kWarps] * a.h_kv;
  if (blockIdx.x == 0) {
    int64_t at = chunk[threadIdx.x];
    for (int b = b_lo; b < b_hi; ++b) {
      a.prefix[b] = at;
      at += seq_units(a, b);
    }
    if (threadIdx.x == 32 * kWarps - 1) a.prefix[a.batch] = chunk[32 * kWarps];
  }
  // sequences with no keys: zeros and -inf
  for (int b = blockIdx.x * kWarps + warp; b < a.batch; b += a.ctas * kWarps) {
    if (seq_units(a, b) > 0) continue;
    const int64_t row = static_cast<int64_t>(b) * a.h_kv * a.G;
    const int n = a.h_kv * a.G;
    for (int i = lane; i < n * D / 8; i += 32) {
      if (a.out_f32) {
        reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * D)[2 * i] = make_float4(0, 0, 0, 0);
        reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * D)[2 * i + 1] = make_float4(0, 0, 0, 0);
      } else {
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * D)[i] = make_uint4(0, 0, 0, 0);
      }
    }
    if (a.lse)
      for (int i = lane; i < n; i += 32) a.lse[row + i] = -INFINITY;
  }

  // this warp's range: consecutive ranges lie on different SMs
  const int nw = static_cast<int>(min(units, static_cast<int64_t>(a.ctas) * kWarps));
  const int wk = warp * a.ctas + blockIdx.x;
  if (wk >= nw) return;
  const int64_t u0 = range_begin(units, wk, nw), u1 = range_begin(units, wk + 1, nw);
  Walk prod;
  {
    int lo = 0, hi = 32 * kWarps - 1;   // last share that begins at or before u0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (chunk[mid] * a.h_kv <= u0) lo = mid; else hi = mid - 1;
    }
    int64_t r = u0 - chunk[lo] * a.h_kv;
    prod.b = lo * per;
    for (;;) {
      prod.n = seq_units(a, prod.b);
      const int64_t all = static_cast<int64_t>(prod.n) * a.h_kv;
      if (r < all) break;
      r -= all;
      ++prod.b;
    }
    prod.g = static_cast<int>(r / prod.n);
    prod.u = static_cast<int>(r - static_cast<int64_t>(prod.g) * prod.n);
    prod.left = u1 - u0;
    walk_piece(a, prod);
  }
  Walk cons = prod;
  const uint32_t ring = smem_u32(smem) + warp * kStages * C::kStage;
  bool more = true;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (more) {
      issue_tile<D, F8>(a, prod, ring + s * C::kStage, lane);
      more = walk_next<C::kTile>(a, prod);
    }
    cp_async_commit();
  }
  State<D, F8> st;
  Query<D, F8> q;
  bool first = true;
  int piece_u = 0;
  for (int slot = 0;; slot = slot == kStages - 1 ? 0 : slot + 1) {
    cp_async_wait_n<kStages - 2>();
    __syncwarp();
    if (more) {
      issue_tile<D, F8>(a, prod, ring + (slot == 0 ? kStages - 1 : slot - 1) * C::kStage, lane);
      more = walk_next<C::kTile>(a, prod);
    }
    cp_async_commit();
    if (first) {
      load_query<D, F8>(q, a.q + (static_cast<int64_t>(cons.b) * a.h_kv + cons.g) * a.G * D, lane, a.G);
      state_clear(st);
      piece_u = cons.u;
    }
    attend_tile<D, F8>(st, q, ring + slot * C::kStage, min(C::kTile, cons.tok_end - cons.u * kUnit), a.scale_log2,
                       lane);
    first = cons.u + C::kTile / kUnit >= cons.ue;
    if (first) {
      const bool from0 = piece_u == 0, to_end = cons.ue == cons.n;
      // a range has at most one piece begun in another range and one that goes on into the next
      write_piece<D, F8>(a, st, cons.b, cons.g, from0 && to_end ? -1 : 2 * wk + (from0 ? 1 : 0), lane);
    }
    if (!walk_next<C::kTile>(a, cons)) break;
  }
}

// Joins the partials of the (sequence, kv head) pairs that several ranges share:
// out = sum_i 2^(lse_i - lse) o_i with lse = log2 sum_i 2^lse_i, pieces in
// ascending order.  WPR warps take one query head's row.  Rows are enumerated
// by pair, or, when there are more pairs than workers, by the worker whose
// range ends inside the pair.
template <int D, int WPR>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args a, int by_pair, int rows) {
  constexpr int LPR = D / 4;            // lanes a piece
  constexpr int GR = 32 * WPR / LPR;    // pieces at a time
  __shared__ float4 acc[WPR > 1 ? GR : 1][LPR];
  const int row = blockIdx.x * (8 / WPR) + (threadIdx.x >> 5) / WPR;
  dec::griddep_wait();
  if (row >= rows) return;
  const int64_t total = a.prefix[a.batch];
  const int64_t units = total * a.h_kv;
  const int nw = static_cast<int>(min(units, static_cast<int64_t>(a.ctas) * kWarps));
  const int h = row % a.G;
  int b, g, wk;
  int64_t s0, s1;
  if (by_pair) {
    b = row / a.G / a.h_kv;
    g = row / a.G - b * a.h_kv;
    const int64_t at = a.prefix[b], n = a.prefix[b + 1] - at;
    if (n == 0) return;
    s0 = at * a.h_kv + g * n;
    s1 = s0 + n;
    wk = static_cast<int>(s0 * nw / units);   // worker of unit s0
    while (range_begin(units, wk, nw) > s0) --wk;
    while (range_begin(units, wk + 1, nw) <= s0) ++wk;
  } else {
    wk = row / a.G;
    if (wk >= nw - 1) return;
    const int64_t u0 = range_begin(units, wk, nw), u1 = range_begin(units, wk + 1, nw);
    int lo = 0, hi = a.batch - 1;             // the sequence of the range's last unit
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.prefix[mid] * a.h_kv <= u1 - 1) lo = mid; else hi = mid - 1;
    }
    b = lo;
    const int64_t first = a.prefix[b] * a.h_kv, n = a.prefix[b + 1] - a.prefix[b];
    g = static_cast<int>((u1 - 1 - first) / n);
    s0 = first + g * n;
    s1 = s0 + n;
    if (s0 < u0) return;                      // begun in an earlier range
  }
  if (s1 <= range_begin(units, wk + 1, nw)) return;   // one piece: written by its warp
  int last = static_cast<int>((s1 - 1) * nw / units);
  while (range_begin(units, last, nw) > s1 - 1) --last;
  while (range_begin(units, last + 1, nw) <= s1 - 1) ++last;
  // piece i: the second slot of wk, then the first slot of wk + i
  const int np = last - wk + 1;
  auto slot = [&](int i) { return static_cast<int64_t>(2 * (wk + i) + (i == 0 ? 1 : 0)) * a.G + h; };
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f;
  for (int i = lane; i < np; i += 32) m = fmaxf(m, a.part_lse[slot(i)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float mr = m == -INFINITY ? 0.f : m;
  for (int i = lane; i < np; i += 32) l += exp2f(a.part_lse[slot(i)] - mr);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int c = threadIdx.x % LPR, r = (threadIdx.x % (32 * WPR)) / LPR;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = r; i < np; i += GR) {
    const float w = exp2f(a.part_lse[slot(i)] - mr) * inv;
    const float4 o = reinterpret_cast<const float4*>(a.part_o + slot(i) * D)[c];
    s.x += w * o.x; s.y += w * o.y; s.z += w * o.z; s.w += w * o.w;
  }
  if (WPR > 1) {   // one row a CTA: no thread of it has returned
    acc[r][c] = s;
    __syncthreads();
    if (r > 0) return;
#pragma unroll
    for (int i = 1; i < GR; ++i) {
      s.x += acc[i][c].x; s.y += acc[i][c].y; s.z += acc[i][c].z; s.w += acc[i][c].w;
    }
  } else if (GR > 1) {
    s.x += __shfl_xor_sync(0xffffffffu, s.x, 16); s.y += __shfl_xor_sync(0xffffffffu, s.y, 16);
    s.z += __shfl_xor_sync(0xffffffffu, s.z, 16); s.w += __shfl_xor_sync(0xffffffffu, s.w, 16);
    if (r > 0) return;
  }
  const int64_t orow = (static_cast<int64_t>(b) * a.h_kv + g) * a.G + h;
  if (a.out_f32) reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * D)[c] = s;
  else
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * D)[c] =
        make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
  if (a.lse && c == 0) a.lse[orow] = l == 0.f ? -INFINITY : m + log2f(l);
}

// workspace layout: prefix, partial log-sum-exps, partial rows
struct Plan {
  size_t off_lse, off_o, bytes;
};
static Plan plan(int batch, int G, int d, int ctas) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t slots = static_cast<size_t>(2) * ctas * kWarps;
  Plan p;
  p.off_lse = up((static_cast<size_t>(batch) + 1) * 8);
  p.off_o = p.off_lse + up(slots * G * 4);
  p.bytes = p.off_o + up(slots * G * d * 4);
  return p;
}

template <int D, bool F8>
static cudaError_t launch(const Args& a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<D, F8>::kSmem);
  if (e != cudaSuccess) return e;
  attend_kernel<D, F8><<<a.ctas, 32 * kWarps, Cfg<D, F8>::kSmem, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  // Few pairs have many pieces each: a CTA a row.  More pairs than SMs: about
  // kWarps pieces or fewer each, a warp a row.
  const int64_t pairs = static_cast<int64_t>(a.batch) * a.h_kv;
  const int64_t workers = static_cast<int64_t>(a.ctas) * kWarps;
  const int rows = static_cast<int>(std::min(pairs, workers) * a.G);
  const bool wide = pairs <= a.ctas;
  cfg.gridDim = dim3(wide ? rows : (rows + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const int by_pair = pairs <= workers;
  return wide ? cudaLaunchKernelEx(&cfg, join_kernel<D, 8>, a, by_pair, rows)
              : cudaLaunchKernelEx(&cfg, join_kernel<D, 1>, a, by_pair, rows);
}

}  // namespace pattn

cudaError_t launch_paged_attn(pattn::Args a, int d, bool f8, void* workspace, cudaStream_t st) {
  const pattn::Plan p = pattn::plan(a.batch, a.G, d, a.ctas);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.prefix = reinterpret_cast<int64_t*>(ws);
  a.part_lse = reinterpret_cast<float*>(ws + p.off_lse);
  a.part_o = reinterpret_cast<float*>(ws + p.off_o);
  if (d == 128) return f8 ? pattn::launch<128, true>(a, st) : pattn::launch<128, false>(a, st);
  return f8 ? pattn::launch<64, true>(a, st) : pattn::launch<64, false>(a, st);
}

}  // namespace infllm2
