// Attention of one new token a sequence over its whole paged key-value cache:
// the dense side of the dense/sparse switch at decode (the sparse side is
// decode.cu).
//
// For query head h of kv group g and the first n = len[b] positions u,
//   z_u = scale log2(e) q_h . k_u,  lse = log2 sum_u 2^z_u,  out = sum_u 2^(z_u - lse) v_u,
// in one pass with a running reference maximum and sum.  Every key and value is
// read once for the group's G <= 16 query heads, so HBM is the bound; 4 d G flop
// a (token, kv head) go to warp-level mma.sync m16n8k16 in the transposed form
//   S^T [16 tokens x 8 heads] = K Q^T,   O^T [16 columns x 8 heads] += V^T P^T,
// so groups of at most 8 heads need half the products of larger ones (NH = 1 or
// 2 tiles of heads).
//
// Split.  Lengths are known on the device only, so the grid is fixed (one CTA
// an SM) and every warp works alone: the tiles of all (sequence, kv head) pairs,
// in order, each pair with one more for its start and end, are cut into equal
// ranges, one a warp, whatever the lengths.  A warp's last piece of a pair meets
// those of the CTA's next warps in shared memory when they belong to the same
// pair; a pair that then lies within one CTA's run of warps is written out, and
// the others leave normalised partials and their log-sum-exps in the workspace,
// at most one a CTA and one more, which a second kernel (programmatic dependent
// launch) joins in ascending order.  Nothing waits on another CTA.
//
// A warp streams tiles of 8 KB (K and V of 16, 32 or 64 tokens) through its own
// kStages-deep cp.async ring, the page numbers of a tile fetched one tile ahead
// of its copies.  Rows past the piece are filled with zeros, not read, so what
// lies in unwritten slots never enters a product.
//
// 8 bits.  K and V go from e4m3 to f16 exactly.  q is scaled to f16 by a power
// of two a head (its 8 significant bits are kept down to 2^-29 of the head's
// largest element, and 2^-39 of it absolutely).  A value's scale multiplies its
// probability: w_u = p_u scale_u c in f16, with c a power of two a head that brings the
// head's largest p_u scale_u so far to 2^11 (2^(11 + kMargin) before c is lowered).
// What counts is p scale and not the scale alone: a large row of no weight
// leaves c as it is, and w keeps 11 bits down to 2^-25 of the head's largest.
//
// Measured (one B200, sustained): 16 x 131072 8-bit, 1.11 GB, 193-215 us (5.1-5.7
// TB/s; 32 heads), 178-181 us with 8 heads a group; 16 x 65536 bf16, 1.07 GB, 175-179 us; 64 bf16
// sequences up to 8192, 0.27 GB, 57 us; one sequence of 1000 10 us.  A tile of the first costs its warp
// 1800 cycles of products and softmax and 750 of copies and bookkeeping, with two warps
// a scheduler.  That fits within the bandwidth at full clocks and not at those which the
// power cap leaves.  More warps (12 x 2 stages), smaller tiles and TMA boxes were slower.
#include "paged_split.cuh"
#include "sm100.cuh"

namespace infllm2 {

namespace pattn {

using dec::cp_async_commit;
using dec::cp_async_wait_n;

constexpr int kStages = 3;
constexpr int kUnit = 16;           // tokens; every page size is a multiple of it
constexpr float kMargin = 4.f;      // a reference is raised only past this many log2 units
constexpr float kTop = 11.f;        // 8 bits: log2 of the weight that the reference stands for
constexpr int kHalf = 4096;         // bytes of K, and of V, in a stage

// The products, the transposed loads and movmatrix are plain (not volatile) asm, so
// the compiler may interleave the chains of a tile; tile_pin keeps them
// between the wait for a tile and the reuse of its slot.
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr));
}
// `bytes` (0 .. 16) from src, zeros after them
__device__ __forceinline__ void cp_async16_part(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16_full(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
// (volatile: issued in program order, all before their first use)
__device__ __forceinline__ void ld_part(float& v, const float* p) {
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
}
__device__ __forceinline__ void ld_part(float4& v, const float* p) {
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
}
// transpose of an 8x8 matrix of 16-bit elements held two a lane
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// two fp32 products in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// (subnormal numbers included)
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pow2_of(float e) { return __int_as_float((static_cast<int>(e) + 127) << 23); }
__device__ __forceinline__ float exponent_of(float p) { return static_cast<float>((__float_as_int(p) >> 23) - 127); }
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
  Join* desc;             // workspace: what to join, by pair or by worker
  float* part_o;          // workspace: [2 * workers][G][D]
  float* part_lse;        // workspace: [2 * workers][G]
  int32_t by_pair;        // at most as many pairs as workers
  int32_t n_pages, page_shift, batch, max_pages, h_kv, G, ctas, out_f32;
  float scale_log2;
};

// tokens of a sequence; a length outside [0, capacity] counts as 0 (recorded by CTA 0)
__device__ __forceinline__ int seq_len(const Args& a, int b) {
  const int n = __ldg(a.len + b);
  const bool ok = n >= 0 && n <= static_cast<int64_t>(a.max_pages) << a.page_shift;
  if (!ok && blockIdx.x == 0) record_status(INFLLM2_ERR_DEVICE_BOUNDS);
  return ok ? n : 0;
}
template <int kTile>
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }
// a pair's share of the ranges
__device__ __forceinline__ int pair_cost(int tiles) { return tiles > 0 ? tiles + 1 : 0; }

template <int D, bool F8>
struct Cfg {
  static constexpr int kRow = F8 ? D : 2 * D;         // bytes a row
  static constexpr int kTile = kHalf / kRow;          // tokens a tile
  static constexpr int CH = kRow / 16;                // 16-byte pieces a row
  static constexpr int kScale = F8 ? 8 * kTile : 0;   // bytes of scales in a stage
  static constexpr int kStage = 2 * kHalf + kScale;
  static constexpr int kSmem = kWarps * kStages * kStage;
  static constexpr int S = kTile / 8;                 // consecutive tokens of a lane group
  static constexpr int MT = kTile / 16;               // 16-token tiles of S^T
  static constexpr int DT = D / 16;                   // 16-column tiles of O^T
};

// Row g + 8h (g < 8, h < 2) of the tile's S^T tile m is its token S g + 2 m + h: the
// order is free (probabilities and values use the same one), and this one gives
// lane group g the S consecutive tokens from S g on, so its scales are vectors.

// Shared-memory byte of 16-byte piece c of the tile's token S g + x.  Rows of 128
// bytes or more have lines of their own, the piece XORed with a number made of
// g; two 64-byte rows (g and g ^ 1) share a line.  The XOR numbers let the eight
// lanes of each shared-memory phase (K: two lane groups' rows, four pieces
// each; V: four rows, two pieces each, or eight rows of an ldmatrix) meet all banks.
template <int CH, int S, bool F8>
__device__ __forceinline__ uint32_t piece_at(int g, int x, int c) {
  if (CH == 4)
    return ((g >> 1) * S + x) * 128 + (((g & 1) ^ ((g >> 1) & 1)) << 6) + ((c ^ ((g >> 2) << 1)) << 4);
  const int f = F8 ? (((g & 1) << 2) ^ (g & 6)) : (((g & 1) << 2) | (g >> 1));
  return (g * S + x) * (CH * 16) + ((c ^ f) << 4);
}

// Walks the tiles of a warp's range.
struct Walk {
  int b, g, n, t, te;   // sequence, kv head, its tiles, the next one, end of this piece
  int len;              // the sequence's tokens
  int64_t left;         // cost of the range from the end of this piece on
  int tok_end;          // tokens of the piece end here
  const int32_t* row;   // the sequence's pages
};

// Takes sequence b.  Its length is read once, and lane 0's is the warp's: the warp's lanes walk together, and nothing
// reads past a sequence's pages, whatever the length does meanwhile.
template <int kTile>
__device__ __forceinline__ void walk_seq(const Args& a, Walk& w) {
  w.len = __shfl_sync(0xffffffffu, seq_len(a, w.b), 0);
  w.n = tiles_of<kTile>(w.len);
}

// the piece of pair (b, g) from cost position y on; false when the range covers none of its tiles
template <int kTile>
__device__ __forceinline__ bool walk_piece(const Args& a, Walk& w, int y) {
  const int take = static_cast<int>(min(static_cast<int64_t>(w.n + 1 - y), w.left));
  w.left -= take;
  w.t = max(y - 1, 0);
  w.te = y + take - 1;
  w.tok_end = min(w.len, w.te * kTile);
  w.row = a.table + static_cast<int64_t>(w.b) * a.max_pages;
  return w.t < w.te;
}

// the first piece after pair (b, g); false when the range is done (or, with lengths that change under the call, when
// there is no further sequence)
template <int kTile>
__device__ __forceinline__ bool walk_pair(const Args& a, Walk& w) {
  if (w.left <= 0) return false;
  if (++w.g == a.h_kv) {
    w.g = 0;
    do {
      if (++w.b >= a.batch) return false;
      walk_seq<kTile>(a, w);
    } while (w.n == 0);
  }
  return walk_piece<kTile>(a, w, 0);   // an empty piece (the pair's start alone) ends its range
}

// to the next tile; false when the range is done
template <int kTile>
__device__ __forceinline__ bool walk_next(const Args& a, Walk& w) {
  return ++w.t < w.te || walk_pair<kTile>(a, w);
}

// The pages of the walk's tile: one where pages hold whole tiles, else one for every 16-token group
// (-1: no token of the piece in it).  Nothing here waits for them.
template <int kTile>
__device__ __forceinline__ void fetch_pages(const Args& a, const Walk& w, int (&page)[kTile / kUnit]) {
  const int tok0 = w.t * kTile;
  page[0] = __ldg(w.row + (tok0 >> a.page_shift));
  if ((kTile >> a.page_shift) > 1) {
#pragma unroll
    for (int i = 1; i < kTile / kUnit; ++i) {
      page[i] = -1;
      if (tok0 + i * kUnit < w.tok_end) page[i] = __ldg(w.row + ((tok0 + i * kUnit) >> a.page_shift));
    }
  }
}

// Instruction i copies the S tokens of lane group i, 512 contiguous bytes, for K
// and for V.  piece_at of the eight differs by i * 512 and an XOR of the lane's
// part with 16 f(i), which takes few values.
template <int D, bool F8>
__device__ __forceinline__ void issue_tile(const Args& a, const Walk& w, const int (&page)[Cfg<D, F8>::kTile / kUnit],
                                           uint32_t stage, int lane) {
  using C = Cfg<D, F8>;
  constexpr int NG = C::kTile / kUnit;   // 16-token groups
  constexpr int IPG = 8 / NG;            // instructions a group
  const int tok0 = w.t * C::kTile;
  const int nv = min(C::kTile, w.tok_end - tok0);
  const int slot0 = tok0 & ((1 << a.page_shift) - 1);
  const bool one = (C::kTile >> a.page_shift) <= 1;
  int pg[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) pg[i] = i == 0 || one ? page[0] : page[i];
  const int r0 = lane / C::CH, c = lane % C::CH;   // instruction i: tokens S i + r0
  int64_t at[NG];                        // first row of the group
  bool ok = nv == C::kTile;
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    at[i] = ((static_cast<int64_t>(pg[i]) * a.h_kv + w.g) << a.page_shift) +
            ((slot0 + i * kUnit) & ((1 << a.page_shift) - 1));
    ok = ok && static_cast<unsigned>(pg[i]) < static_cast<unsigned>(a.n_pages);
  }
  if (ok) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint8_t* k = a.k_pages + (at[g] * C::kRow + lane * 16);
      const uint8_t* v = a.v_pages + (at[g] * C::kRow + lane * 16);
#pragma unroll
      for (int j = 0; j < IPG; ++j) {
        const int i = g * IPG + j;
        const uint32_t dst = stage + piece_at<C::CH, C::S, F8>(i, r0, c);
        cp_async16_full(dst, k + j * 512);
        cp_async16_full(dst + kHalf, v + j * 512);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = C::S * i + r0 < nv, good = static_cast<unsigned>(pg[i / IPG]) < static_cast<unsigned>(a.n_pages);
      if (in && !good) record_status(INFLLM2_ERR_DEVICE_BOUNDS);
      const int64_t off = in && good ? at[i / IPG] * C::kRow + (i % IPG) * 512 + lane * 16 : 0;
      const uint32_t dst = stage + piece_at<C::CH, C::S, F8>(i, r0, c);
      cp_async16_part(dst, a.k_pages + off, in && good ? 16 : 0);
      cp_async16_part(dst + kHalf, a.v_pages + off, in && good ? 16 : 0);
    }
  }
  if constexpr (F8) {
    // scales: pieces of four tokens, K's then V's
    constexpr int P = C::kTile / 4;
    if (lane < 2 * P) {
      const int t = 4 * (lane % P);
      int64_t row = at[0];
      int of = pg[0];
#pragma unroll
      for (int i = 1; i < NG; ++i)
        if (t / kUnit == i) { row = at[i]; of = pg[i]; }
      const bool good = static_cast<unsigned>(of) < static_cast<unsigned>(a.n_pages);
      const int bytes = good ? max(0, min(16, 4 * (nv - t))) : 0;
      const float* src = lane < P ? a.k_scale : a.v_scale;
      cp_async16_part(stage + 2 * kHalf + lane * 16, bytes > 0 ? src + row + (t & (kUnit - 1)) : src, bytes);
    }
  }
}

// Query heads as B fragments (head gid + 8 nh): bf16 as they are, or (F8) f16
// scaled to [2^14, 2^15) by a power of two a head; `unscale` (of this lane's
// score columns, heads 2 tig + e + 8 nh) undoes it and carries the softmax scale.
template <int D, bool F8, int NH>
struct Query {
  uint32_t b[NH][D / 16][2];
  float s[NH][2];
};

template <int D, bool F8, int NH>
__device__ __forceinline__ void load_query(Query<D, F8, NH>& f, const __nv_bfloat16* q, int lane, int G,
                                           float scale_log2) {
  const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int nh = 0; nh < NH; ++nh) {
    const int h = gid + 8 * nh;
    if (!F8) {
      // pieces of 8: k steps 2j and 2j + 1 cover d = 8 (tig + 4j) + {0, 1, 2, 3} and + {4, 5, 6, 7} in this lane
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const uint4 v = h < G ? *reinterpret_cast<const uint4*>(q + h * D + 8 * (tig + 4 * j)) : make_uint4(0, 0, 0, 0);
        f.b[nh][2 * j][0] = v.x; f.b[nh][2 * j][1] = v.y;
        f.b[nh][2 * j + 1][0] = v.z; f.b[nh][2 * j + 1][1] = v.w;
      }
      f.s[nh][0] = f.s[nh][1] = scale_log2;
      continue;
    }
    // pieces of 16: k step 4j + i covers d = 16 (tig + 4j) + 4i + {0, 1, 2, 3} in this lane
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
    // bf16 exponent e: |q| < 2^(e - 126); scaled by 2^(141 - e)
    const int e = min(max(static_cast<int>(top >> 7), 15), 254);
    const float up = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
    const float un = __uint_as_float(static_cast<uint32_t>(e - 14) << 23) * scale_log2;
    f.s[nh][0] = __shfl_sync(0xffffffffu, un, 8 * tig);
    f.s[nh][1] = __shfl_sync(0xffffffffu, un, 8 * tig + 4);
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4& x = v[2 * j + (i >> 1)];
        const uint32_t w0 = (i & 1) ? x.z : x.x, w1 = (i & 1) ? x.w : x.y;
        f.b[nh][4 * j + i][0] = pack_f16(__uint_as_float(w0 << 16) * up, __uint_as_float(w0 & 0xffff0000u) * up);
        f.b[nh][4 * j + i][1] = pack_f16(__uint_as_float(w1 << 16) * up, __uint_as_float(w1 & 0xffff0000u) * up);
      }
  }
}

// This lane's columns: heads 2 tig + e + 8 nh.
template <int D, bool F8, int NH>
struct State {
  float o[NH][D / 16][4];   // O^T tiles: rows gid and gid + 8
  float m[NH][2];           // reference maximum, log2 units (the same in all lanes of a head)
  float l[NH][2];           // this lane's share of the sum
  float c[NH][2];           // F8: the weights' factor, 2^(kTop + m - (log2 of the reference p scale))
  float lim[NH][2];         // F8: log2 of the weight, without c, past which the reference is raised
};

template <int D, bool F8, int NH>
__device__ __forceinline__ void state_clear(State<D, F8, NH>& s) {
#pragma unroll
  for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) s.o[nh][i][0] = s.o[nh][i][1] = s.o[nh][i][2] = s.o[nh][i][3] = 0.f;
    s.m[nh][0] = s.m[nh][1] = -INFINITY;
    s.l[nh][0] = s.l[nh][1] = 0.f;
    s.c[nh][0] = s.c[nh][1] = 1.f;
    s.lim[nh][0] = s.lim[nh][1] = -INFINITY;
  }
}

template <int D, bool F8, int NH>
__device__ __forceinline__ void attend_tile(State<D, F8, NH>& st, const Query<D, F8, NH>& q, uint32_t stage, int nv,
                                            int lane) {
  using C = Cfg<D, F8>;
  const int gid = lane >> 2, tig = lane & 3;
  float z[C::MT][NH][4];
  // S^T = K Q^T
#pragma unroll
  for (int m = 0; m < C::MT; ++m) {
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) z[m][nh][0] = z[m][nh][1] = z[m][nh][2] = z[m][nh][3] = 0.f;
#pragma unroll
    for (int j = 0; j < C::CH / 4; ++j) {
      const uint4 k0 = lds128(stage + piece_at<C::CH, C::S, F8>(gid, 2 * m, tig + 4 * j));
      const uint4 k1 = lds128(stage + piece_at<C::CH, C::S, F8>(gid, 2 * m + 1, tig + 4 * j));
      if (F8) {
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t f[4] = {paged::e4m3x2_to_f16x2(static_cast<uint16_t>(w0[i])),
                                 paged::e4m3x2_to_f16x2(static_cast<uint16_t>(w1[i])),
                                 paged::e4m3x2_to_f16x2(static_cast<uint16_t>(w0[i] >> 16)),
                                 paged::e4m3x2_to_f16x2(static_cast<uint16_t>(w1[i] >> 16))};
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) mma<true>(z[m][nh], f, q.b[nh][4 * j + i][0], q.b[nh][4 * j + i][1]);
        }
      } else {
        const uint32_t f0[4] = {k0.x, k1.x, k0.y, k1.y}, f1[4] = {k0.z, k1.z, k0.w, k1.w};
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
          mma<false>(z[m][nh], f0, q.b[nh][2 * j][0], q.b[nh][2 * j][1]);
          mma<false>(z[m][nh], f1, q.b[nh][2 * j + 1][0], q.b[nh][2 * j + 1][1]);
        }
      }
    }
  }
  // the keys' scales; the values' scales
  float vs[F8 ? C::S : 1];
  if constexpr (F8) {
    float ks[C::S];
#pragma unroll
    for (int i = 0; i < C::S / 4; ++i) {
      const uint4 k = lds128(stage + 2 * kHalf + 4 * C::S * gid + 16 * i);
      const uint4 v = lds128(stage + 2 * kHalf + 4 * C::kTile + 4 * C::S * gid + 16 * i);
      ks[4 * i] = __uint_as_float(k.x); ks[4 * i + 1] = __uint_as_float(k.y);
      ks[4 * i + 2] = __uint_as_float(k.z); ks[4 * i + 3] = __uint_as_float(k.w);
      vs[4 * i] = __uint_as_float(v.x); vs[4 * i + 1] = __uint_as_float(v.y);
      vs[4 * i + 2] = __uint_as_float(v.z); vs[4 * i + 3] = __uint_as_float(v.w);
    }
    // Scores in log2 units.  q's factor comes first: a product is below 2^31 (448 d 2^15), and times a large scale
    // it would overflow before a small factor brings it down.  Two factors a score cost 8 instructions a tile and eight
    // heads in packed form; the other way, smaller key scales where one is past 2^96, is a branch in every tile (16 x
    // 131072 212.4 us packed, 214.1 with the branch).
#pragma unroll
    for (int m = 0; m < C::MT; ++m)
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = ks[2 * m + h];
          const float2 y = mul2(mul2(make_float2(z[m][nh][2 * h], z[m][nh][2 * h + 1]),
                                     make_float2(q.s[nh][0], q.s[nh][1])), make_float2(x, x));
          z[m][nh][2 * h] = y.x;
          z[m][nh][2 * h + 1] = y.y;
        }
  }
  if (nv < C::kTile) {
#pragma unroll
    for (int m = 0; m < C::MT; ++m)
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (C::S * gid + 2 * m + (e >> 1) >= nv) z[m][nh][e] = -INFINITY;
  }
  // Raise a reference where a score (F8: or a score with its value's scale) passes it.  The second is
  // bounded by the lane's largest score and largest scale, which differ little over a few consecutive tokens.
  float top[NH][2], vtop = -INFINITY;
  if constexpr (F8) {
    vtop = 0.f;
#pragma unroll
    for (int i = 0; i < C::S; ++i) vtop = fmaxf(vtop, fabsf(vs[i]));
    vtop = lg2(vtop);
  }
  bool past = false;
#pragma unroll
  for (int nh = 0; nh < NH; ++nh)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float t = -INFINITY;
#pragma unroll
      for (int m = 0; m < C::MT; ++m) t = fmaxf(t, fmaxf(z[m][nh][e], z[m][nh][2 + e]));
      top[nh][e] = F8 ? t : t * q.s[nh][e];
      past = past || top[nh][e] > st.m[nh][e] + kMargin;
      if constexpr (F8) past = past || top[nh][e] + vtop > st.lim[nh][e];
    }
  if (__any_sync(0xffffffffu, past)) {
    float lv[F8 ? C::S : 1];
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < C::S; ++i) lv[i] = lg2(fabsf(vs[i]));
    }
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = top[nh][e];
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
        // (F8: whole log2 units, so that factors are powers of two)
        const float m = fmaxf(st.m[nh][e], F8 ? ceilf(t) : t);
        const float f = st.m[nh][e] == m ? 1.f : ex2(st.m[nh][e] - m);
        float back = f;
        if constexpr (F8) {
          float y = -INFINITY;
#pragma unroll
          for (int k = 0; k < C::MT; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) y = fmaxf(y, z[k][nh][2 * h + e] + lv[2 * k + h]);
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
          y = fmaxf(st.lim[nh][e] - kMargin, ceilf(y));
          // c, 1 / c and 1 / (l c) stay normal numbers (m = -inf, where nothing has a weight yet: any c)
          const float was = exponent_of(st.c[nh][e]), now = fminf(fmaxf(kTop + m - y, -118.f), 104.f);
          back = ex2((st.m[nh][e] == m ? 0.f : st.m[nh][e] - m) + (now - was));
          st.c[nh][e] = pow2_of(now);
          st.lim[nh][e] = m + (kTop + kMargin - now);
        }
        st.m[nh][e] = m;
        st.l[nh][e] *= f;
#pragma unroll
        for (int i = 0; i < C::DT; ++i) {
          st.o[nh][i][e] *= back;
          st.o[nh][i][2 + e] *= back;
        }
      }
  }
  // Probabilities as B fragments: w in f16, or P in bf16 twice, its upper half and
  // what that leaves (together 2^-15; one bf16 alone would add its 2^-8 to the output's
  // own, for 1-2 % of the time: 57.0 against 58.2 us for 64 sequences up to 8192).  (A second f16
  // part of w changes the third digit of a bf16 output's error and takes 235 us for 207 at 16 x
  // 131072.)  The sums of both stay in fp32 unrounded.  Both parts of a P above 0 are above 0 (the upper half is cut off, not
  // rounded, and 2^-22 P added to the rest), so an infinite value gives that infinity twice and never
  // inf - inf or 0 inf.
  float neg[NH][2];
#pragma unroll
  for (int nh = 0; nh < NH; ++nh)
#pragma unroll
    for (int e = 0; e < 2; ++e) neg[nh][e] = st.m[nh][e] == -INFINITY ? 0.f : -st.m[nh][e];
  uint32_t p[C::MT][NH][2], rest[C::MT][NH][2];   // 16 tokens x 8 heads
#pragma unroll
  for (int m = 0; m < C::MT; ++m)
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = ex2(F8 ? z[m][nh][e] + neg[nh][e & 1] : fmaf(z[m][nh][e], q.s[nh][e & 1], neg[nh][e & 1]));
        st.l[nh][e & 1] += w[e];
      }
      if constexpr (F8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = vs[2 * m + h];
          const float2 y = mul2(mul2(make_float2(w[2 * h], w[2 * h + 1]), make_float2(x, x)),
                                make_float2(st.c[nh][0], st.c[nh][1]));
          w[2 * h] = y.x;
          w[2 * h + 1] = y.y;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x = F8 ? pack_f16(w[2 * h], w[2 * h + 1])
                              : __byte_perm(__float_as_uint(w[2 * h]), __float_as_uint(w[2 * h + 1]), 0x7632);
        p[m][nh][h] = movmatrix(x);
        if (!F8) {
          constexpr float kUp = 1.f + 1.f / (1 << 22);
          rest[m][nh][h] = movmatrix(pack_bf16(fmaf(w[2 * h], kUp, -__uint_as_float(x << 16)),
                                               fmaf(w[2 * h + 1], kUp, -__uint_as_float(x & 0xffff0000u))));
        }
      }
    }
  // O^T += V^T P^T
  const uint32_t vb = stage + kHalf;
#pragma unroll
  for (int m = 0; m < C::MT; ++m) {
    if (F8) {
      // bytes of four rows: column D/8 gid + 2 i + {0, 1} is row gid, gid + 8 of O^T's tile i
      constexpr int W = D / 32;   // words a row and lane
      uint32_t w[4][W];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int g = 2 * tig + (i & 1), x = 2 * m + (i >> 1);
        if (W == 4) {
          const uint4 v = lds128(vb + piece_at<C::CH, C::S, F8>(g, x, gid));
          w[i][0] = v.x; w[i][1] = v.y; w[i][W - 2] = v.z; w[i][W - 1] = v.w;
        } else {
          const uint2 v = lds64(vb + piece_at<C::CH, C::S, F8>(g, x, gid >> 1) + (gid & 1) * 8);
          w[i][0] = v.x; w[i][1] = v.y;
        }
      }
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t lo = __byte_perm(w[0][j], w[1][j], e ? 0x7362 : 0x5140);
          const uint32_t hi = __byte_perm(w[2][j], w[3][j], e ? 0x7362 : 0x5140);
          const uint32_t f[4] = {paged::e4m3x2_to_f16x2(static_cast<uint16_t>(lo)),
                                 paged::e4m3x2_to_f16x2(static_cast<uint16_t>(lo >> 16)),
                                 paged::e4m3x2_to_f16x2(static_cast<uint16_t>(hi)),
                                 paged::e4m3x2_to_f16x2(static_cast<uint16_t>(hi >> 16))};
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) mma<true>(st.o[nh][2 * j + e], f, p[m][nh][0], p[m][nh][1]);
        }
    } else {
      // four 8x8 matrices: columns 0-7 and 8-15 of the tile, rows 0-7, then rows 8-15 of the step
      const int i = lane >> 3;
#pragma unroll
      for (int j = 0; j < C::DT; ++j) {
        uint32_t f[4];
        ldsm_x4_t(f, vb + piece_at<C::CH, C::S, F8>(lane & 7, 2 * m + (i >> 1), 2 * j + (i & 1)));
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) mma<false>(st.o[nh][j], f, p[m][nh][0], p[m][nh][1]);
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) mma<false>(st.o[nh][j], f, rest[m][nh][0], rest[m][nh][1]);
      }
    }
  }
}

// Nothing that reads the tile moves past this point: its results are needed here.
template <int D, bool F8, int NH>
__device__ __forceinline__ void tile_pin(State<D, F8, NH>& st) {
#pragma unroll
  for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      asm volatile("" : "+f"(st.o[nh][i][0]), "+f"(st.o[nh][i][1]), "+f"(st.o[nh][i][2]), "+f"(st.o[nh][i][3])::"memory");
    asm volatile("" : "+f"(st.l[nh][0]), "+f"(st.l[nh][1])::"memory");
  }
}

// Floats from one row of a partial in shared memory to the next: the lanes of a store (rows by tig, columns by
// gid) then meet all banks.
template <int D>
constexpr int kPartLd = D + 4;

// A row's sum over the lanes that share it: the factor that normalises O^T, and the log-sum-exp.
// l = 0: every score was -inf; the row is empty.
template <int D, bool F8, int NH>
__device__ __forceinline__ void row_stats(const State<D, F8, NH>& st, int nh, int e, float& inv, float& lse) {
  float l = st.l[nh][e];
  l += __shfl_xor_sync(0xffffffffu, l, 4);
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
  inv = l == 0.f ? 0.f : 1.f / (F8 ? l * st.c[nh][e] : l);
  lse = l == 0.f ? -INFINITY : st.m[nh][e] + log2f(l);
}

// The normalised rows of all 8 NH heads (of which G are real) to shared memory, then their log-sum-exps.  Kept apart
// from write_piece: every warp runs this once, from a cold instruction cache, so it is short.
template <int D, bool F8, int NH>
__device__ __forceinline__ void keep_piece(const State<D, F8, NH>& st, float* mine, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int nh = 0; nh < NH; ++nh)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float inv, lse;
      row_stats(st, nh, e, inv, lse);
      float* row = mine + (8 * nh + 2 * tig + e) * kPartLd<D>;
      if (gid == 0) mine[8 * NH * kPartLd<D> + 8 * nh + 2 * tig + e] = lse;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        // F8: columns D/8 gid + 2 i + {0, 1}; else 16 i + gid + {0, 8}
        const float v0 = st.o[nh][i][e] * inv, v1 = st.o[nh][i][2 + e] * inv;
        if (F8) {
          *reinterpret_cast<float2*>(row + D / 8 * gid + 2 * i) = make_float2(v0, v1);
        } else {
          row[16 * i + gid] = v0;
          row[16 * i + 8 + gid] = v1;
        }
      }
    }
}

// The G heads' normalised rows and log-sum-exps to the pair's rows of the output (`out`) or to partial `slot`.
template <int D, bool F8, int NH>
__device__ __forceinline__ void write_piece(const Args& a, const State<D, F8, NH>& st, bool out, int pair,
                                            int64_t slot, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int nh = 0; nh < NH; ++nh)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float inv, lse;
      row_stats(st, nh, e, inv, lse);
      const int h = 2 * tig + e + 8 * nh;
      if (h >= a.G) continue;
      const int64_t row = (out ? pair : slot) * a.G + h;
      const bool b16 = out && !a.out_f32;
      float* po = (!out ? a.part_o : static_cast<float*>(a.out)) + row * D;
      __nv_bfloat16* pb = static_cast<__nv_bfloat16*>(a.out) + row * D;
      if (gid == 0 && (!out || a.lse)) (out ? a.lse : a.part_lse)[row] = lse;
      if (F8) {
        // columns D/8 gid .. D/8 (gid + 1)
#pragma unroll
        for (int i = 0; i < D / 16; i += 2) {
          const float v0 = st.o[nh][i][e] * inv, v1 = st.o[nh][i][2 + e] * inv;
          const float v2 = st.o[nh][i + 1][e] * inv, v3 = st.o[nh][i + 1][2 + e] * inv;
          const int d = D / 8 * gid + 2 * i;
          if (!b16) *reinterpret_cast<float4*>(po + d) = make_float4(v0, v1, v2, v3);
          else *reinterpret_cast<uint2*>(pb + d) = make_uint2(pack_bf16(v0, v1), pack_bf16(v2, v3));
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float v = st.o[nh][i][2 * r + e] * inv;
            const int d = 16 * i + 8 * r + gid;
            if (!b16) po[d] = v;
            else pb[d] = __float2bfloat16_rn(v);
          }
      }
    }
}

template <int D, bool F8, int NH>
__global__ void __launch_bounds__(32 * kWarps, 1) attend_kernel(const __grid_constant__ Args a) {
  using C = Cfg<D, F8>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t chunk[32 * kWarps + 1];   // cost before each thread's share of the sequences
  __shared__ int4 info[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  dec::griddep_launch_dependents();

  // cost of all sequences
  const int per = (a.batch + 32 * kWarps - 1) / (32 * kWarps);
  const int b_lo = min(a.batch, static_cast<int>(threadIdx.x) * per), b_hi = min(a.batch, b_lo + per);
  int64_t incl = 0;
  for (int b = b_lo; b < b_hi; ++b) incl += pair_cost(tiles_of<C::kTile>(seq_len(a, b)));
  incl *= a.h_kv;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) chunk[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int64_t c = chunk[w];
    if (w < warp) before += c;
    total += c;
  }
  __syncthreads();
  chunk[threadIdx.x + 1] = before + incl;
  if (threadIdx.x == 0) chunk[0] = 0;
  __syncthreads();
  // sequences with no keys: zeros and -inf
  for (int b = blockIdx.x * kWarps + warp; b < a.batch; b += a.ctas * kWarps) {
    if (seq_len(a, b) > 0) continue;
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
    if (a.by_pair)
      for (int i = lane; i < a.h_kv; i += 32) a.desc[static_cast<int64_t>(b) * a.h_kv + i] = Join{0, 0, -1, 0};
  }

  // this warp's range
  const int wk = blockIdx.x * kWarps + warp;
  const int64_t share = div_pos(total + a.ctas * kWarps - 1, a.ctas * kWarps);
  const int64_t x0 = min(total, share * wk), x1 = min(total, x0 + share);
  Walk prod;
  bool more = x0 < x1;
  if (more) {
    // the last share of sequences that begins at or before x0: among every kWarps-th, then next to it
    int lo = 31 - __clz(__ballot_sync(0xffffffffu, chunk[lane * kWarps] <= x0));
    lo *= kWarps;
    lo += 31 - __clz(__ballot_sync(0xffffffffu, lane < kWarps && chunk[lo + lane] <= x0));
    int64_t r = x0 - chunk[lo];
    int64_t cost = 1;
    prod.b = lo * per;
    for (; prod.b < a.batch; ++prod.b) {
      walk_seq<C::kTile>(a, prod);
      cost = pair_cost(prod.n);
      if (r < cost * a.h_kv) break;
      r -= cost * a.h_kv;
    }
    more = prod.b < a.batch;   // (lengths that change under the call)
    prod.g = more ? static_cast<int>(div_pos(r, cost)) : 0;
    prod.left = x1 - x0;
    more = more && (walk_piece<C::kTile>(a, prod, static_cast<int>(r - prod.g * cost)) || walk_pair<C::kTile>(a, prod));
  }
  Walk cons = prod;
  const uint32_t ring = smem_u32(smem) + warp * kStages * C::kStage;
  int page[C::kTile / kUnit];
  if (more) fetch_pages<C::kTile>(a, prod, page);
  State<D, F8, NH> st;
  Query<D, F8, NH> q;
  bool first = true, run = more;
  int t0 = 0, pieces = 0, rest = 0;
  int4 last = make_int4(-1, 0, 0, 0);   // the last piece: its pair, from the start?, to the end?, the only one?
  // iteration i copies tile i into its slot and attends to tile i - (kStages - 1)
  for (int i = 0, slot = 0; run; ++i, slot = slot == kStages - 1 ? 0 : slot + 1) {
    if (more) {
      issue_tile<D, F8>(a, prod, page, ring + slot * C::kStage, lane);
      more = walk_next<C::kTile>(a, prod);
      if (more) fetch_pages<C::kTile>(a, prod, page);
    }
    cp_async_commit();
    if (i < kStages - 1) continue;
    if (first) {
      load_query<D, F8, NH>(q, a.q + (static_cast<int64_t>(cons.b) * a.h_kv + cons.g) * a.G * D, lane, a.G,
                            a.scale_log2);
      state_clear(st);
      t0 = cons.t;
    }
    cp_async_wait_n<kStages - 1>();
    __syncwarp();
    uint32_t stage = ring + (slot == kStages - 1 ? 0 : slot + 1) * C::kStage;
    asm volatile("" : "+r"(stage)::"memory");   // the tile's loads stay behind the wait
    attend_tile<D, F8, NH>(st, q, stage, min(C::kTile, cons.tok_end - cons.t * C::kTile), lane);
    tile_pin(st);
    __syncwarp();
    first = cons.t + 1 == cons.te;
    if (first) {
      const int pair = cons.b * a.h_kv + cons.g;
      const bool from0 = t0 == 0;
      last = make_int4(pair, from0, cons.te == cons.n, pieces++ == 0);
      rest = cons.n - cons.te;
      // the range's last piece waits in this warp's share of the ring; an earlier one ends its pair
      const bool keep = cons.left <= 1;   // (what is left is no other pair's tile)
      if (keep)
        keep_piece<D, F8, NH>(st, reinterpret_cast<float*>(smem + warp * kStages * C::kStage), lane);
      else
        write_piece<D, F8, NH>(a, st, from0, pair, 2 * static_cast<int64_t>(wk), lane);
      if (!keep && from0 && a.by_pair && lane == 0) a.desc[pair] = Join{0, 0, -1, 0};
    }
    run = walk_next<C::kTile>(a, cons);
  }
  cp_async_wait_n<0>();
  if (lane == 0) info[warp] = last;
  __syncthreads();
  // Runs of warps whose last pieces are of one pair: the CTA's threads share a
  // run's rows, four columns a thread.
  constexpr int kWarpFloats = kStages * C::kStage / 4;
  for (int w0 = 0, w1; w0 < kWarps; w0 = w1 + 1) {
    const int4 head = info[w0];
    w1 = w0;
    if (head.x < 0) continue;
    int4 tail = head;
    while (w1 < kWarps - 1) {
      const int4 next = info[w1 + 1];
      if (next.x != head.x || !next.w) break;
      tail = next;
      ++w1;
    }
    const bool out = head.y && tail.z;
    const float* part = reinterpret_cast<const float*>(smem) + w0 * kWarpFloats;
    const int len = w1 - w0 + 1;
    const int64_t row0 = (out ? head.x : 2 * static_cast<int64_t>(blockIdx.x * kWarps + w0) + (head.y ? 1 : 0)) * a.G;
    for (int i = threadIdx.x; i < a.G * (D / 4); i += 32 * kWarps) {
      const int h = i / (D / 4), at4 = h * (kPartLd<D> / 4) + i % (D / 4);
      float4 o = reinterpret_cast<const float4*>(part)[at4];
      float lse = part[8 * NH * kPartLd<D> + h];
      if (len > 1) {
        float x[kWarps], m = lse;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          x[w] = part[min(w, len - 1) * kWarpFloats + 8 * NH * kPartLd<D> + h];
          m = fmaxf(m, x[w]);
        }
        const float ref = m == -INFINITY ? 0.f : m;
        float l = ex2(lse - ref);
        o.x *= l; o.y *= l; o.z *= l; o.w *= l;
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
          if (w < len) {
            const float f = ex2(x[w] - ref);
            const float4 v = reinterpret_cast<const float4*>(part + w * kWarpFloats)[at4];
            l += f;
            o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
          }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
        lse = l == 0.f ? -INFINITY : m + log2f(l);
      }
      const int64_t at = row0 * (D / 4) + i;
      if (!out) reinterpret_cast<float4*>(a.part_o)[at] = o;
      else if (a.out_f32) reinterpret_cast<float4*>(a.out)[at] = o;
      else reinterpret_cast<uint2*>(a.out)[at] = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
      if (i % (D / 4) == 0 && (!out || a.lse)) (out ? a.lse : a.part_lse)[row0 + h] = lse;
    }
    if (warp == w0 && lane == 0) {   // its first warp describes a run
      Join joins{0, 0, -1, 0};
      if (head.y && !tail.z) joins = describe_join(wk, head.x, x1, rest, share, total, a.ctas);
      if (!a.by_pair) a.desc[wk] = joins;
      else if (head.y) a.desc[head.x] = joins;
    }
    if (!a.by_pair && lane == 0 && warp > w0 && warp <= w1) a.desc[wk] = Join{0, 0, -1, 0};
  }
  if (!a.by_pair && last.x < 0 && lane == 0) a.desc[wk] = Join{0, 0, -1, 0};
}

// Joins the partials of the (sequence, kv head) pairs that several ranges share:
// out = sum_i 2^(lse_i - lse) o_i with lse = log2 sum_i 2^lse_i, pieces in
// ascending order.  WPR warps take one query head's row.  Rows are enumerated
// by pair, or, when there are more pairs than workers, by the worker whose
// range the pair begins in.
template <int D, int WPR>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args a, int rows) {
  constexpr int LPR = D / 4;            // lanes a piece
  constexpr int GR = 32 * WPR / LPR;    // pieces at a time
  constexpr int RPC = 8 / WPR;          // rows a CTA
  __shared__ float4 acc_s[RPC][WPR > 1 ? GR : 1][LPR];
  __shared__ float2 stat_s[RPC][WPR > 1 ? GR : 1];
  auto& acc = acc_s[(threadIdx.x >> 5) / WPR];
  auto& stat = stat_s[(threadIdx.x >> 5) / WPR];
  const int row = blockIdx.x * RPC + (threadIdx.x >> 5) / WPR;
  const int at = row / a.G, h = row - at * a.G;
  dec::griddep_wait();
  if (row >= rows) return;
  const Join d = a.desc[at];
  if (d.ctas == 0) return;              // written by its warps
  if (!join_in_bounds(d, a.batch * a.h_kv, a.ctas)) {   // (lengths that changed under the call)
    if (threadIdx.x % 32 == 0) record_status(INFLLM2_ERR_DEVICE_BOUNDS);
    return;
  }
  const int np = join_pieces(d), pair = d.pair;
  auto slot = [&](int i) { return static_cast<int64_t>(join_slot(d, i)) * a.G + h; };
  const int c = threadIdx.x % LPR, r = (threadIdx.x % (32 * WPR)) / LPR;
  // this thread's pieces with a running maximum, eight loads in flight
  float m = -INFINITY, l = 0.f;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = r; i0 < np; i0 += 8 * GR) {
    float4 o[8];
    float x[8];
    float top = m;
#pragma unroll
    for (int j = 0; j < 8; ++j) {   // past the last piece: that piece again, without weight
      const int64_t at = slot(min(i0 + j * GR, np - 1));
      ld_part(x[j], a.part_lse + at);
      ld_part(o[j], a.part_o + at * D + 4 * c);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (i0 + j * GR >= np) x[j] = -INFINITY;
      top = fmaxf(top, x[j]);
    }
    const float ref = top == -INFINITY ? 0.f : top;
    const float f = exp2f(m - ref);
    l *= f; s.x *= f; s.y *= f; s.z *= f; s.w *= f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (i0 + j * GR >= np) break;
      const float w = exp2f(x[j] - ref);
      l += w;
      s.x += w * o[j].x; s.y += w * o[j].y; s.z += w * o[j].z; s.w += w * o[j].w;
    }
    m = top;
  }
  // the groups' sums
  if (WPR > 1) {   // all warps of a row come here or none
    acc[r][c] = s;
    if (c == 0) stat[r] = make_float2(m, l);
    if (WPR == 8) __syncthreads();
    else named_bar_sync(1 + (threadIdx.x >> 5) / WPR, 32 * WPR);
    if (r > 0) return;
    float top = m;
#pragma unroll
    for (int i = 1; i < GR; ++i) top = fmaxf(top, stat[i].x);
    const float ref = top == -INFINITY ? 0.f : top;
    const float f = exp2f(m - ref);
    l *= f; s.x *= f; s.y *= f; s.z *= f; s.w *= f;
#pragma unroll
    for (int i = 1; i < GR; ++i) {
      const float w = exp2f(stat[i].x - ref);
      l += w * stat[i].y;
      s.x += w * acc[i][c].x; s.y += w * acc[i][c].y; s.z += w * acc[i][c].z; s.w += w * acc[i][c].w;
    }
    m = top;
  } else if (GR > 1) {
    const float top = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
    const float f = exp2f(m - (top == -INFINITY ? 0.f : top));
    l *= f; s.x *= f; s.y *= f; s.z *= f; s.w *= f;
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    s.x += __shfl_xor_sync(0xffffffffu, s.x, 16); s.y += __shfl_xor_sync(0xffffffffu, s.y, 16);
    s.z += __shfl_xor_sync(0xffffffffu, s.z, 16); s.w += __shfl_xor_sync(0xffffffffu, s.w, 16);
    if (r > 0) return;
    m = top;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  s.x *= inv; s.y *= inv; s.z *= inv; s.w *= inv;
  const int64_t orow = static_cast<int64_t>(pair) * a.G + h;
  if (a.out_f32) reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * D)[c] = s;
  else
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * D)[c] =
        make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
  if (a.lse && c == 0) a.lse[orow] = l == 0.f ? -INFINITY : m + log2f(l);
}

// workspace layout: descriptors, partial log-sum-exps, partial rows
struct Plan {
  size_t off_lse, off_o, bytes;
};
static Plan plan(int G, int d, int ctas) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t slots = static_cast<size_t>(2) * ctas * kWarps;
  Plan p;
  p.off_lse = up(slots / 2 * sizeof(Join));   // pairs (at most workers), or workers
  p.off_o = p.off_lse + up(slots * G * 4);
  p.bytes = p.off_o + up(slots * G * d * 4);
  return p;
}

template <int D, bool F8, int NH>
static cudaError_t launch_heads(const Args& a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, F8, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<D, F8>::kSmem);
  if (e != cudaSuccess) return e;
  attend_kernel<D, F8, NH><<<a.ctas, 32 * kWarps, Cfg<D, F8>::kSmem, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  // A warp joins 8 pieces (16 for d = 64) at a time: one warp a row where pairs have
  // few (at most CTAs / pairs and two, on average), else four or a CTA, so
  // that rows of a few times the average take one round.
  const int64_t pairs = static_cast<int64_t>(a.batch) * a.h_kv;
  const int64_t workers = static_cast<int64_t>(a.ctas) * kWarps;
  const int rows = static_cast<int>(std::min(pairs, workers) * a.G);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  if (pairs * 8 < a.ctas) {
    cfg.gridDim = dim3(rows);
    return cudaLaunchKernelEx(&cfg, join_kernel<D, 8>, a, rows);
  }
  if (pairs < a.ctas) {
    cfg.gridDim = dim3((rows + 1) / 2);
    return cudaLaunchKernelEx(&cfg, join_kernel<D, 4>, a, rows);
  }
  cfg.gridDim = dim3((rows + 7) / 8);
  return cudaLaunchKernelEx(&cfg, join_kernel<D, 1>, a, rows);
}

template <int D, bool F8>
static cudaError_t launch(const Args& a, cudaStream_t st) {
  return a.G > 8 ? launch_heads<D, F8, 2>(a, st) : launch_heads<D, F8, 1>(a, st);
}

}  // namespace pattn

cudaError_t launch_paged_attn(pattn::Args a, int d, bool f8, void* workspace, cudaStream_t st) {
  const pattn::Plan p = pattn::plan(a.G, d, a.ctas);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.desc = reinterpret_cast<pattn::Join*>(ws);
  a.by_pair = static_cast<int64_t>(a.batch) * a.h_kv <= static_cast<int64_t>(a.ctas) * pattn::kWarps;
  a.part_lse = reinterpret_cast<float*>(ws + p.off_lse);
  a.part_o = reinterpret_cast<float*>(ws + p.off_o);
  if (d == 128) return f8 ? pattn::launch<128, true>(a, st) : pattn::launch<128, false>(a, st);
  return f8 ? pattn::launch<64, true>(a, st) : pattn::launch<64, false>(a, st);
}

}  // namespace infllm2
