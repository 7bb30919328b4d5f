// attention_rows.cu -- attention of few query rows per head (single tokens of a
// few branches) over the packed cache, decoded straight into the operands of
// register-level matrix products: nothing but the packed fields crosses HBM.
//
// Bound by the decoding's latency, not by memory and by no single pipe: at 40 heads x
// 37440 tokens x 128 channels the packed fields are 162 MB (25 us), while every element
// takes about four instructions to rebuild, not counting what each group of them needs;
// one row takes 225 us, eight 234 us and sixteen 245 us (at rank 16 292, 301 and 311),
// with 56 % of the issue slots and 44 % of the integer pipe in use by the 12 warps that
// the registers leave an SM.  So the layout serves the decoder.  A warp takes 16
// keys at a time; in the products' operand layout (lane = 4 g + c) the channels
// are permuted such that a lane owns a quarter head of keys g and g + 8 of K'
// (whole code words) and D / 8 channels of keys 2c, 2c+1, 2c+8, 2c+9 of V', and
// each decoded pair goes from the conversion into its product without passing
// through shared memory.
//
//   K'  = bf16((c + mn + code sc) + cs sum_i U_i c8_i).  The compensation is a
//         product too: c8 is exact in bf16, and U is split into three bf16 parts
//         (24 bits), kept in shared memory in operand order.
//   S   = Q K'^T, P = 2^(scale log2e S - m), O += P V': m16n8k16, rows = queries.
//
// Each CTA takes an equal run of (head, 16-key tile) positions, whatever the
// number of heads, and gives one partial per head it touches.  Its warps take
// tiles in turn, each with a running maximum, sum and O and a small ring of
// asynchronous copies of its own, and meet at the end of a head and where the
// basis or table version changes: U and, when both fit (C D <= 32768), the
// centroid tables of the version at hand lie in shared memory (larger tables are
// read through the cache).
#include <math.h>

#include "around.cuh"
#include "dequant_pairs.cuh"
#include "tc.cuh"

namespace qwm {
namespace {
using namespace tc;

constexpr int NW_ROWS = 12;    // warps of the attention: 168 registers per thread, and 32 to 48 bytes
                               // of spills at head 128 (16 warps spill much more: 320 us, against
                               // 240 us when this was chosen)
constexpr int NW_UNPACK = 16;  // and of the unpacking, which keeps no O
constexpr int KT = 16;        // keys per tile
constexpr int NSTAGE = 2;     // tiles in a warp's ring
constexpr float TAU = 8.0f;   // a row's reference moves when its maximum grew by more (log2)

struct RowsArgs {
  Dims Dm;
  CacheView v;
  int64_t T;
  const uint16_t* Q;
  int64_t ldq;
  int rows, Hq, g;     // rows per head: tokens x query heads of a key head, 16 at most
  float scale_log2;
  float *ws_o, *ws_l;  // [slot][token][Hq][D], [slot][token][Hq]
  int64_t nq;
  int nslot;           // slots of a head
  int64_t nt, total;   // tiles per head, in all
};

template <int D>
struct Stage {  // its fixed fields: code words and K's parameters
  static constexpr uint32_t KC = 0, VC = KC + KT * D / 4, KP = VC + KT * D / 4;
};
// Shared memory.  A stage holds the packed fields of a tile; where each begins
// depends on the rank, the group size and the centroid numbers' width.
// RK: the rank, rounded up to 8 or 16 (the depth of the compensation's products).
template <int D, int NW, int RK>
struct RLay {
  static constexpr uint32_t OFF_ML = 0;                        // [warp][16] m, l
  static constexpr uint32_t OFF_Q = OFF_ML + 2 * NW * 16 * 4;  // [16][D] bf16
  static constexpr uint32_t OFF_U = OFF_Q + 16 * D * 2;        // [D / 8][32] parts of U
  static constexpr uint32_t OFF_ST = OFF_U + D / 8 * 32 * (RK == 8 ? 16 : 24);  // [warp][NSTAGE] stages
};
// Place of the low parts of U behind the others (RK = 16).
template <int D>
__host__ __device__ constexpr uint32_t u_low() { return D / 8 * 32 * 16; }
// The warps' O of rows_kernel, over the tables' place.
template <int D>
constexpr uint32_t merge_bytes() { return NW_ROWS * 16 * D * 4; }
struct Fields {  // offsets in a stage
  uint32_t vp, co, cs, ki, vi, stage, tab;  // and of the tables (or the warps' O) in shared memory
};
template <int D, int NW, int RK>
__host__ __device__ __forceinline__ Fields fields_of(const Dims& Dm) {
  using L = RLay<D, NW, RK>;
  Fields f;
  f.vp = Stage<D>::KP + KT * Dm.ng * 4;
  f.co = f.vp + KT * Dm.ng * 4;
  f.cs = f.co + KT * Dm.r;
  f.ki = f.cs + KT * 2;
  f.vi = f.ki + KT * Dm.idx_bytes;
  f.stage = f.vi + KT * Dm.idx_bytes;
  f.tab = (L::OFF_ST + NW * NSTAGE * f.stage + 127) / 128 * 128;
  return f;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), bf16; with 8 in place of 16; and D = A B.
__device__ __forceinline__ void mma16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0));
}

// The CTA whose run holds position x.
__device__ __forceinline__ int64_t cta_of(const RowsArgs& A, int64_t x) {
  return ((x + 1) * gridDim.x - 1) / A.total;
}

// What a lane copies of every tile of a head, 16 bytes a piece: code words of K
// and V, parameters (K in the lower half warp, V in the upper; at 8 groups a
// second piece each), and one piece of the short fields.  (Capacities are
// multiples of 128 keys, so whole tiles lie in the buffers.)
template <int D>
struct Source {
  const uint8_t *codes, *params, *rest;  // of tile 0; codes of K, V at + vcodes
  int64_t vcodes;
  uint32_t dst_params, dst_rest, step_rest;
};

template <int D>
__device__ __forceinline__ Source<D> source_of(const Dims& Dm, const Fields& F, const PackedHead& p) {
  using L = Stage<D>;
  const int lane = threadIdx.x & 31, r = Dm.r, ib = Dm.idx_bytes;
  Source<D> S;
  S.codes = p.k_codes + 16 * lane;
  S.vcodes = p.v_codes - p.k_codes;
  // a tile has 4 ng pieces of parameters for K and as many for V
  const int half = lane >> 4, i = lane & 15;
  S.params = (const uint8_t*)(half ? p.v_params : p.k_params) + 16 * i;
  S.dst_params = (half ? F.vp : L::KP) + 16 * i;
  // the short ones side by side: at most 16 + 2 + 2 + 2 lanes
  const int a = r, b = a + 2, c = b + ib, d = c + ib;  // ends, in pieces
  S.rest = nullptr;
  S.dst_rest = S.step_rest = 0;
  auto piece = [&](const void* src, uint32_t dst, int first, int bytes) {
    S.rest = (const uint8_t*)src + 16 * (lane - first);
    S.dst_rest = dst + 16 * (lane - first);
    S.step_rest = KT * bytes;
  };
  if (lane < a) piece(p.k_coef, F.co, 0, r);
  else if (lane < b) piece(p.k_cscale, F.cs, a, 2);
  else if (lane < c) piece(p.k_idx, F.ki, b, ib);
  else if (lane < d) piece(p.v_idx, F.vi, c, ib);
  return S;
}

// Start copying tile t into the stage at `st`.
template <int D>
__device__ __forceinline__ void fill_stage(const Source<D>& S, int ng, uint32_t st, int64_t t) {
  using L = Stage<D>;
  const int lane = threadIdx.x & 31;
  if (16 * lane < KT * D / 4) {
    const uint8_t* src = S.codes + t * (KT * D / 4);
    cp_async16_cg(st + L::KC + 16 * lane, src);
    cp_async16_cg(st + L::VC + 16 * lane, src + S.vcodes);
  }
  const uint8_t* par = S.params + t * (KT * 4 * ng);
  if ((lane & 15) < 4 * ng) cp_async16_cg(st + S.dst_params, par);
  if (ng > 4) cp_async16_cg(st + S.dst_params + 256, par + 256);
  if (S.rest) cp_async16_cg(st + S.dst_rest, S.rest + t * S.step_rest);
}

// The first position in (at, end) whose versions are not those of `at`, or end
// (versions never fall along the cache); 32 probes at a time, one warp.
__device__ __forceinline__ int64_t versions_end(const CacheView& v, int64_t at, int64_t end) {
  const int lane = threadIdx.x & 31;
  const int tv = v.tokver[at], cv = v.centver[at];
  int64_t lo = at, hi = end;  // position lo has them; hi is end or has not
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 31) / 32, x = lo + (lane + 1) * step;
    const bool same = x < hi && v.tokver[x] == tv && v.centver[x] == cv;
    const int n = __popc(__ballot_sync(0xffffffffu, same));  // the first n probes
    const int64_t up = lo + (n + 1) * step;
    lo += n * step;
    hi = up < hi ? up : hi;
  }
  return hi;
}

// What a warp keeps while it works on one head.
template <int D>
struct State {
  float o[D / 8][4];      // O: n-tile j holds channels g' D/8 + j; rows g, g + 8
  float m0, m1, l0, l1;   // reference and (this lane's part of the) sum of rows g, g + 8
};

// A lane's K channels are c D/4 ..; of the two code words that they fill at D =
// 128, lanes with c >= 2 take the second first, so that the four lanes of a key
// read centroid pieces of different banks.  Channel of position e (0 .. D/4 - 1).
template <int D>
__device__ __forceinline__ int k_channel(int c, int e) {
  return c * (D / 4) + (D == 128 ? e ^ (8 * (c & 2)) : e);
}

// U of head h, version ver, as B operands: n-tile j's column n is position
// 2j + n % 2 of the lanes with c = n / 2.  A lane's pairs of components, 2c and 2c + 1
// (and 2c + 8, 2c + 9), as {high, middle, low, -}, or {high, high, middle, middle}
// and {low, low}.
template <int D, int RK>
__device__ __forceinline__ void stage_basis(const Dims& Dm, const CacheView& v, uint8_t* dst, int h,
                                            int ver) {
  const int r = Dm.r;
  const float* U = basis_of(v, Dm, ver, h);
  for (int e = threadIdx.x; e < D / 8 * 32; e += blockDim.x) {
    const int j = e >> 5, g = (e & 31) >> 2, c = e & 3;
    const float* u = U + (size_t)k_channel<D>(g >> 1, 2 * j + (g & 1)) * r + 2 * c;
    uint32_t part[RK / 8][3];
#pragma unroll
    for (int i = 0; i < RK / 8; ++i) {
      const int at = 2 * c + 8 * i;
      float x = at < r ? __ldg(u + 8 * i) : 0.0f, y = at + 1 < r ? __ldg(u + 8 * i + 1) : 0.0f;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        part[i][k] = pack_bf16(x, y);
        x -= __uint_as_float(part[i][k] << 16);  // exact: the rounding's remainder
        y -= __uint_as_float(part[i][k] & 0xffff0000u);
      }
    }
    if constexpr (RK == 8) {
      reinterpret_cast<uint4*>(dst)[e] = make_uint4(part[0][0], part[0][1], part[0][2], 0);
    } else {
      reinterpret_cast<uint4*>(dst)[e] = make_uint4(part[0][0], part[1][0], part[0][1], part[1][1]);
      reinterpret_cast<uint2*>(dst + u_low<D>())[e] = make_uint2(part[0][2], part[1][2]);
    }
  }
}

__device__ __forceinline__ uint32_t i8_pair_bf16(uint32_t two) {
  return pack_bf16(i8_to_f32((int8_t)(two & 0xff)), i8_to_f32((int8_t)(two >> 8)));
}

// A lane's coefficients of key k: components 2c, 2c + 1 (and 2c + 8, 2c + 9), as an A operand.
template <int RK>
__device__ __forceinline__ void coefs_of(const uint8_t* co, int k, int c, int r, uint32_t (&a)[RK / 8]) {
#pragma unroll
  for (int i = 0; i < RK / 8; ++i) {
    const int at = 2 * c + 8 * i;
    uint32_t two = 0;
    if (r == RK) {
      two = *reinterpret_cast<const uint16_t*>(co + k * RK + at);
    } else {
      if (at < r) two = co[k * r + at];
      if (at + 1 < r) two |= (uint32_t)co[k * r + at + 1] << 8;
    }
    a[i] = i8_pair_bf16(two);
  }
}

// sum_i U_i c8_i of keys g and g + 8 (a[0], a[1]) over n-tile j, from the lane's place
// in the staged basis.
template <int D, int RK>
__device__ __forceinline__ void compensation(float (&d)[4], const uint32_t (&a)[2][RK / 8],
                                             const uint8_t* us, int j) {
  const uint4 u = *reinterpret_cast<const uint4*>(us + 16 * (threadIdx.x & 31) + j * 512);
  if constexpr (RK == 8) {  // (the high and middle parts as one product of depth 16)
    mma16_new(d, a[0][0], a[1][0], a[0][0], a[1][0], u.x, u.y);
    mma8(d, a[0][0], a[1][0], u.z);
  } else {
    const uint2 l = *reinterpret_cast<const uint2*>(us + u_low<D>() + 8 * (threadIdx.x & 31) + j * 256);
    mma16_new(d, a[0][0], a[1][0], a[0][1], a[1][1], u.x, u.y);
    mma16(d, a[0][0], a[1][0], a[0][1], a[1][1], u.z, u.w);
    mma16(d, a[0][0], a[1][0], a[0][1], a[1][1], l.x, l.y);
  }
}

// S_i and M_i of one parameter word (positions 0 .. 3 of a code byte).  Scalar
// fp32 here: the two-wide forms need their operands in register pairs, and the
// moves that gather them cost more than they save (399 against 328 us with 8 warps
// at the size above).
struct Decode {
  float s[4], m[4];
};
__device__ __forceinline__ Decode decode_of(uint32_t par) {
  const float mn = h2f((uint16_t)(par & 0xffffu)), sc = h2f((uint16_t)(par >> 16));
  Decode d;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    d.s[i] = sc * (float)(256 >> (2 * i));
    d.m[i] = mn - d.s[i];
  }
  return d;
}

// (x & mask of position P) | 1.0f in one instruction; `one` holds 0x3F800000.
template <int P>
__device__ __forceinline__ float magic(uint32_t x, uint32_t one) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(x), "n"(3u << (15 + 2 * P)), "r"(one));
  return __uint_as_float(d);
}
__device__ __forceinline__ float magic(uint32_t x, int p, uint32_t one) {
  return p == 0 ? magic<0>(x, one) : p == 1 ? magic<1>(x, one) : p == 2 ? magic<2>(x, one) : magic<3>(x, one);
}

// The code byte b of word w at bits 15 .. 22.
template <int B>
__device__ __forceinline__ uint32_t code_byte(uint32_t w) {
  return B == 0 ? w << 15 : B == 1 ? w << 7 : B == 2 ? w >> 1 : w >> 9;
}

// Rows of the staged tables: 16-byte pieces exchanged by the row number, so that
// the keys of a warp, whose rows are as good as random, spread over the banks.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
  return (uint32_t)row * (D * 2) + ((uint32_t)(piece ^ (row & 7)) << 4);
}

// One warp: keys [lo, hi) of the staged 16, all of the staged basis and table
// version (the fields of other keys are not used).
template <int D, bool TAB, int RK>
__device__ __forceinline__ void keys16(const RowsArgs& A, const Fields& F, const uint8_t* pk,
                                       const uint8_t* smem,
                                       const uint16_t* gk, const uint16_t* gv, int lo, int hi,
                                       State<D>& st) {
  using L = RLay<D, NW_ROWS, RK>;
  using St = Stage<D>;
  constexpr int KCH = D / 4;       // a lane's K channels
  constexpr int KW = KCH / 16;     // their code words
  constexpr int VCH = D / 8;       // a lane's V channels
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const Dims& Dm = A.Dm;
  const int gs = Dm.G == 16 ? 4 : 5;  // log2 of the group size
  const int ng = Dm.ng, r = Dm.r, ib = Dm.idx_bytes;
  const uint8_t* tk = smem + F.tab;
  const uint8_t* tvv = tk + Dm.C * D * 2;
  auto number = [&](uint32_t fields, int k, bool live) {  // centroid (0 of a key not worked on)
    return !live ? 0 : ib == 1 ? (int)pk[fields + k] : (int)reinterpret_cast<const uint16_t*>(pk + fields)[k];
  };

  uint32_t one;
  asm volatile("mov.b32 %0, 0x3F800000;" : "=r"(one));

  // ---- K' of keys g and g + 8, and S
  float s[2][4];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[x][e] = 0.0f;
  {
    int row[2];
    float cs[2];
    uint32_t a[2][RK / 8];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int k = g + 8 * x;
      const bool live = k >= lo && k < hi;
      row[x] = number(F.ki, k, live);
      cs[x] = 0.0f;
      if (r > 0) {
        cs[x] = live ? h2f(reinterpret_cast<const uint16_t*>(pk + F.cs)[k]) : 0.0f;
        coefs_of<RK>(pk + F.co, k, c, r, a[x]);
      }
    }
    const uint8_t* us = smem + L::OFF_U;
    const uint4* qs = reinterpret_cast<const uint4*>(smem + L::OFF_Q) + lane;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const int wa = D == 128 ? w ^ (c >> 1) : w;  // the lane's code word
      uint32_t code[2];
      Decode gc[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int k = g + 8 * x;
        code[x] = reinterpret_cast<const uint32_t*>(pk + St::KC)[k * (D / 16) + c * KW + wa];
        gc[x] = decode_of(reinterpret_cast<const uint32_t*>(pk + St::KP)[k * ng + ((c * KCH + 16 * wa) >> gs)]);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {  // 8 channels: a piece of the centroid
        uint4 cw[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int piece = c * (KCH / 8) + 2 * wa + hf;
          cw[x] = TAB ? *reinterpret_cast<const uint4*>(tk + piece_at<D>(row[x], piece))
                      : __ldg(reinterpret_cast<const uint4*>(gk + (size_t)row[x] * D) + piece);
        }
#pragma unroll
        for (int q4 = 0; q4 < 2; ++q4) {  // 4 channels: a step of 16 over the warp
          const int ks = 4 * w + 2 * hf + q4;
          uint32_t b[2][2], bytes[2];
#pragma unroll
          for (int x = 0; x < 2; ++x)
            bytes[x] = hf == 0 ? (q4 == 0 ? code_byte<0>(code[x]) : code_byte<1>(code[x]))
                               : (q4 == 0 ? code_byte<2>(code[x]) : code_byte<3>(code[x]));
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int j = 2 * ks + y;
            float corr[4];
            if (r > 0) compensation<D, RK>(corr, a, us, j);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t at = bytes[x];
              const uint32_t cb = reinterpret_cast<const uint32_t(&)[4]>(cw[x])[2 * q4 + y];
              float v0 = __uint_as_float(cb << 16) + fmaf(magic(at, 2 * y, one), gc[x].s[2 * y], gc[x].m[2 * y]);
              float v1 = __uint_as_float(cb & 0xffff0000u) +
                         fmaf(magic(at, 2 * y + 1, one), gc[x].s[2 * y + 1], gc[x].m[2 * y + 1]);
              if (r > 0) {
                v0 = fmaf(corr[2 * x], cs[x], v0);
                v1 = fmaf(corr[2 * x + 1], cs[x], v1);
              }
              b[x][y] = pack_bf16(v0, v1);
            }
          }
          const uint4 q = qs[ks * 32];  // rows g and g + 8, the same four channels
          mma16(s[0], q.x, q.y, q.z, q.w, b[0][0], b[0][1]);
          mma16(s[1], q.x, q.y, q.z, q.w, b[1][0], b[1][1]);
        }
      }
    }
  }

  // ---- softmax: this lane's keys 2c, 2c + 1 (s[0]) and 8 + 2c, 9 + 2c (s[1])
  uint32_t p[4];
  {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = 8 * x + 2 * c + e;
        const bool live = k >= lo && k < hi;
        s[x][e] = live ? s[x][e] * A.scale_log2 : -INFINITY;
        s[x][2 + e] = live ? s[x][2 + e] * A.scale_log2 : -INFINITY;
      }
    float t0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
    float t1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
    if (__any_sync(0xffffffffu, t0 > st.m0 + TAU || t1 > st.m1 + TAU)) {
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, o));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, o));
      }
      // (some key of the 16 is worked on, so the new references are finite)
      const float n0 = fmaxf(t0, st.m0), n1 = fmaxf(t1, st.m1);
      const float f0 = ex2(st.m0 - n0), f1 = ex2(st.m1 - n1);
      st.m0 = n0;
      st.m1 = n1;
      st.l0 *= f0;
      st.l1 *= f1;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        st.o[j][0] *= f0;
        st.o[j][1] *= f0;
        st.o[j][2] *= f1;
        st.o[j][3] *= f1;
      }
    }
    float w[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      w[x][0] = ex2(s[x][0] - st.m0);
      w[x][1] = ex2(s[x][1] - st.m0);
      w[x][2] = ex2(s[x][2] - st.m1);
      w[x][3] = ex2(s[x][3] - st.m1);
      st.l0 += w[x][0] + w[x][1];
      st.l1 += w[x][2] + w[x][3];
    }
    p[0] = pack_bf16(w[0][0], w[0][1]);  // weights to bf16: 2^-8 relative at most
    p[1] = pack_bf16(w[0][2], w[0][3]);
    p[2] = pack_bf16(w[1][0], w[1][1]);
    p[3] = pack_bf16(w[1][2], w[1][3]);
  }

  // ---- V' of keys 2c, 2c + 1, then of 2c + 8, 2c + 9, and O
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    int row[2];
    uint32_t code[2];
    float mn[2], sc[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = 2 * c + 8 * x + e;
      const bool live = k >= lo && k < hi;
      row[e] = number(F.vi, k, live);
      const uint8_t* cd = pk + St::VC + k * (D / 4) + g * (VCH / 4);
      code[e] = VCH == 16 ? *reinterpret_cast<const uint32_t*>(cd) : *reinterpret_cast<const uint16_t*>(cd);
      // a key that is not worked on: finite (its weight is 0)
      const uint32_t par = live ? reinterpret_cast<const uint32_t*>(pk + F.vp)[k * ng + (g * VCH >> gs)] : 0u;
      mn[e] = h2f((uint16_t)(par & 0xffffu));
      sc[e] = h2f((uint16_t)(par >> 16));
    }
    uint64_t S[4], M[4];  // of both keys, for the position in the code byte
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = (float)(256 >> (2 * i));
      S[i] = fmul2(f2pack(sc[0], sc[1]), f2pack(f, f));
      M[i] = fsub2(f2pack(mn[0], mn[1]), S[i]);
    }
#pragma unroll
    for (int j8 = 0; j8 < VCH / 8; ++j8) {
      uint4 cw[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int piece = g * (VCH / 8) + j8;
        cw[e] = TAB ? *reinterpret_cast<const uint4*>(tvv + piece_at<D>(row[e], piece))
                    : __ldg(reinterpret_cast<const uint4*>(gv + (size_t)row[e] * D) + piece);
      }
      uint32_t bytes[2];
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        const int j = 8 * j8 + jj;
        if (jj % 4 == 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            bytes[e] = j / 4 == 0   ? code_byte<0>(code[e])
                       : j / 4 == 1 ? code_byte<1>(code[e])
                       : j / 4 == 2 ? code_byte<2>(code[e])
                                    : code_byte<3>(code[e]);
        }
        float mm[2], cc[2], v0, v1;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mm[e] = magic(bytes[e], j % 4, one);
          const uint32_t q = reinterpret_cast<const uint32_t(&)[4]>(cw[e])[jj / 2];
          cc[e] = __uint_as_float(jj & 1 ? q & 0xffff0000u : q << 16);
        }
        f2unpack(fadd2(f2pack(cc[0], cc[1]), ffma2(f2pack(mm[0], mm[1]), S[j % 4], M[j % 4])), v0, v1);
        mma8(st.o[j], p[2 * x], p[2 * x + 1], pack_bf16(v0, v1));
      }
    }
  }
}

// The head's table rows into shared memory, loads four deep.
template <int D>
__device__ __forceinline__ void stage_tables(const Dims& Dm, uint8_t* d, const uint16_t* gk,
                                             const uint16_t* gv) {
  constexpr int P = D / 8;  // pieces per row
  const uint32_t tb = Dm.C * D * 2;
  const int n = Dm.C * P, nt = blockDim.x;
  for (int e0 = threadIdx.x; e0 < n; e0 += 4 * nt) {
    uint4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = e0 + u * nt < n ? e0 + u * nt : e0;
      a[u] = __ldg(reinterpret_cast<const uint4*>(gk) + e);
      b[u] = __ldg(reinterpret_cast<const uint4*>(gv) + e);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = e0 + u * nt;
      if (e >= n) break;
      const uint32_t at = piece_at<D>(e / P, e % P);
      *reinterpret_cast<uint4*>(d + at) = a[u];
      *reinterpret_cast<uint4*>(d + tb + at) = b[u];
    }
  }
}

// All warps of a CTA: tokens [at, tend) of head h, span by span of the same
// versions, whose basis and tables are staged; one(pk, lo, hi, t, gk, gv) for each
// tile, warp by warp: keys [lo, hi) of tile t with its fields at pk; gk, gv: the
// head's tables in memory.
template <int D, int NW, bool TAB, int RK, class One>
__device__ __forceinline__ void walk(const Dims& Dm, const CacheView& v, const Fields& F, uint8_t* smem,
                                     int h, int64_t at, int64_t tend, One one) {
  using L = RLay<D, NW, RK>;
  const int warp = threadIdx.x >> 5;
  uint8_t* const ring = smem + L::OFF_ST + warp * NSTAGE * F.stage;
  const uint32_t ring_at = smem_u32(ring);
  const Source<D> src = source_of<D>(Dm, F, packed_head(v, Dm, h));
  int tabver = -1, uver = -1;
  const uint16_t *gk = nullptr, *gv = nullptr;
  while (at < tend) {
    const int uv = v.tokver[at], cvn = v.centver[at];
    const int64_t to = versions_end(v, at, tend);
    // a tile on the border of two spans is worked on in both
    const int64_t first = at / KT + warp, last = (to + KT - 1) / KT;
#pragma unroll
    for (int i = 0; i < NSTAGE - 1; ++i) {
      if (first + i * NW < last) fill_stage<D>(src, Dm.ng, ring_at + i * F.stage, first + i * NW);
      cp_async_commit();
    }
    if (cvn != tabver || uv != uver) {
      __syncthreads();
      if (uv != uver && Dm.r > 0) stage_basis<D, RK>(Dm, v, smem + L::OFF_U, h, uv);
      if (cvn != tabver) {
        const size_t off = (size_t)cvn * cent_slot_elems(Dm) + (size_t)h * Dm.C * D;
        gk = v.cent_k + off;
        gv = v.cent_v + off;
        if (TAB) stage_tables<D>(Dm, smem + F.tab, gk, gv);
      }
      uver = uv;
      tabver = cvn;
      __syncthreads();
    }
    int s = 0;
    for (int64_t t = first; t < last; t += NW) {
      cp_async_wait<NSTAGE - 2>();
      __syncwarp();  // the tile is there; the stage before it is free
      const int64_t ahead = t + (NSTAGE - 1) * NW;
      const int sa = s == 0 ? NSTAGE - 1 : s - 1;
      if (ahead < last) fill_stage<D>(src, Dm.ng, ring_at + sa * F.stage, ahead);
      cp_async_commit();
      const int64_t k0 = t * KT;
      one(ring + s * F.stage, (int)(at > k0 ? at - k0 : 0), (int)(to - k0 < KT ? to - k0 : KT), t, gk, gv);
      s = s + 1 == NSTAGE ? 0 : s + 1;
    }
    cp_async_wait<0>();
    __syncwarp();
    at = to;
  }
}

template <int D, bool TAB, int RK>
__global__ void __launch_bounds__(32 * NW_ROWS, 1) rows_kernel(const __grid_constant__ RowsArgs A) {
  constexpr int NW = NW_ROWS;
  using L = RLay<D, NW, RK>;
  extern __shared__ __align__(128) uint8_t smem[];
  const Dims& Dm = A.Dm;
  const Fields F = fields_of<D, NW, RK>(Dm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t x0 = blockIdx.x * A.total / gridDim.x, x1 = (blockIdx.x + 1) * A.total / gridDim.x;
  State<D> st;
  for (int64_t x = x0; x < x1;) {
    const int h = (int)(x / A.nt);
    const int64_t head0 = (int64_t)h * A.nt, head_end = head0 + A.nt;
    const int64_t end = head_end < x1 ? head_end : x1;
    // ---- this head's Q rows (operand order: four channels of rows g and g + 8 per lane)
    __syncthreads();  // the last head's tables, O and Q are done with
    for (int e = threadIdx.x; e < (D / 16) * 32; e += 32 * NW) {
      const int ks = e >> 5, gg = (e & 31) >> 2, cc = e & 3;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = gg + 8 * y;
        uint2 q = make_uint2(0, 0);
        if (r < A.rows) {
          const int tok = r / A.g;
          q = __ldg(reinterpret_cast<const uint2*>(A.Q + tok * A.ldq + (h * A.g + (r - tok * A.g)) * D +
                                                   k_channel<D>(cc, 4 * ks)));
        }
        reinterpret_cast<uint32_t*>(smem + L::OFF_Q)[e * 4 + y] = q.x;
        reinterpret_cast<uint32_t*>(smem + L::OFF_Q)[e * 4 + 2 + y] = q.y;
      }
    }
    st.m0 = st.m1 = -INFINITY;
    st.l0 = st.l1 = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[j][e] = 0.0f;
    const int64_t at = (x - head0) * KT;
    const int64_t tend = (end - head0) * KT < A.T ? (end - head0) * KT : A.T;
    walk<D, NW, TAB, RK>(Dm, A.v, F, smem, h, at, tend,
                     [&](const uint8_t* pk, int lo, int hi, int64_t, const uint16_t* gk, const uint16_t* gv) {
                       keys16<D, TAB, RK>(A, F, pk, smem, gk, gv, lo, hi, st);
                     });
    x = end;
    // ---- the warps' results: maxima and sums, then O over the tables' place
    float* ml = reinterpret_cast<float*>(smem + L::OFF_ML);
    float* ow = reinterpret_cast<float*>(smem + F.tab);
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
      st.l0 += __shfl_xor_sync(0xffffffffu, st.l0, o);
      st.l1 += __shfl_xor_sync(0xffffffffu, st.l1, o);
    }
    __syncthreads();  // the tables are read
    if (c == 0) {
      ml[warp * 16 + g] = st.m0;
      ml[warp * 16 + g + 8] = st.m1;
      ml[NW * 16 + warp * 16 + g] = st.l0;
      ml[NW * 16 + warp * 16 + g + 8] = st.l1;
    }
    // a lane's n-tile j holds columns 2c, 2c + 1: channels (2c + e) D/8 + j
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        ow[(warp * 16 + g + 8 * (e >> 1)) * D + (2 * c + (e & 1)) * (D / 8) + j] = st.o[j][e];
    __syncthreads();
    const int slot = (int)(blockIdx.x - cta_of(A, head0));
    for (int e = threadIdx.x; e < 16 * D; e += 32 * NW) {
      const int row = e / D, ch = e % D;
      if (row >= A.rows) break;  // rows ascend
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) top = fmaxf(top, ml[w * 16 + row]);
      float l = 0.0f, o = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float m = ml[w * 16 + row];
        const float f = m > -INFINITY ? ex2(m - top) : 0.0f;
        l = fmaf(f, ml[NW * 16 + w * 16 + row], l);
        o = fmaf(f, ow[(w * 16 + row) * D + ch], o);
      }
      const int tok = row / A.g;
      const int64_t out = (int64_t)tok * A.Hq + h * A.g + (row - tok * A.g);
      A.ws_o[((size_t)slot * A.nq * A.Hq + out) * D + ch] = o / l;
      if (ch == 0) {
        A.ws_l[(size_t)slot * A.nq * A.Hq + out] = (top + log2f(l)) * 0.6931471805599453f;
        // the head's last run says which slots stay empty
        if (end == head_end)
          for (int k = slot + 1; k < A.nslot; ++k) A.ws_l[(size_t)k * A.nq * A.Hq + out] = -INFINITY;
      }
    }
  }
}

// ------------------------------------------------------------------ unpacking
// K' and V' of heads h0 .. as [head][T][D] bf16, the cache that the
// reconstruction returns, with the decoding of K' above for both: a lane rebuilds
// 16 adjacent channels of a key at a time and stores them as one 32-byte sector.
// Bound by the decoding as well: 211 us at 40 heads x 37440 tokens x 128 (the 767 MB
// that it writes are 117 us; a thread per 16 channels, with the basis read from
// shared memory for every element, took 700 us); 23 us over 12 x 7919 tokens, where a
// warp has two or three tiles and a block's beginning is not hidden.
struct UnpackArgs {
  Dims Dm;
  CacheView v;
  int64_t T, nt, total;  // tokens; tiles per head, in all
  int h0;
  uint16_t *K, *V;
};

__device__ __forceinline__ void store32(uint16_t* dst, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

template <int D, bool TAB, int RK>
__device__ __forceinline__ void unpack16(const UnpackArgs& A, const Fields& F, const uint8_t* pk,
                                         const uint8_t* smem, const uint16_t* gk, const uint16_t* gv,
                                         int lo, int hi, uint16_t* K, uint16_t* V) {
  using St = Stage<D>;
  constexpr int KCH = D / 4, KW = KCH / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const Dims& Dm = A.Dm;
  const int gs = Dm.G == 16 ? 4 : 5;  // log2 of the group size
  const int ng = Dm.ng, r = Dm.r, ib = Dm.idx_bytes;
  const uint8_t* tk = smem + F.tab;
  const uint8_t* tvv = tk + Dm.C * D * 2;
  uint32_t one;
  asm volatile("mov.b32 %0, 0x3F800000;" : "=r"(one));
  uint32_t a[2][RK / 8];
  float cs[2] = {0.0f, 0.0f};
  bool live[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int k = g + 8 * x;
    live[x] = k >= lo && k < hi;
    if (r > 0) {
      cs[x] = h2f(reinterpret_cast<const uint16_t*>(pk + F.cs)[k]);
      coefs_of<RK>(pk + F.co, k, c, r, a[x]);
    }
  }
  const uint8_t* us = smem + RLay<D, NW_UNPACK, RK>::OFF_U;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const bool comp = kv == 0 && r > 0;
    int row[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t f = kv ? F.vi : F.ki;
      row[x] = !live[x] ? 0
               : ib == 1 ? (int)pk[f + g + 8 * x]
                         : (int)reinterpret_cast<const uint16_t*>(pk + f)[g + 8 * x];
    }
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const int wa = D == 128 ? w ^ (c >> 1) : w;  // the lane's code word
      uint32_t out[2][8];
      uint32_t code[2];
      Decode dc[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int k = g + 8 * x;
        code[x] = reinterpret_cast<const uint32_t*>(pk + (kv ? St::VC : St::KC))[k * (D / 16) + c * KW + wa];
        dc[x] = decode_of(
            reinterpret_cast<const uint32_t*>(pk + (kv ? F.vp : St::KP))[k * ng + ((c * KCH + 16 * wa) >> gs)]);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint4 cw[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int piece = c * (KCH / 8) + 2 * wa + hf;
          cw[x] = TAB ? *reinterpret_cast<const uint4*>((kv ? tvv : tk) + piece_at<D>(row[x], piece))
                      : __ldg(reinterpret_cast<const uint4*>((kv ? gv : gk) + (size_t)row[x] * D) + piece);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {  // pair of channels 2y, 2y + 1 of the piece
          const int j = 8 * w + 4 * hf + y;
          float corr[4];
          if (comp) compensation<D, RK>(corr, a, us, j);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t at = hf == 0 ? (y < 2 ? code_byte<0>(code[x]) : code_byte<1>(code[x]))
                                        : (y < 2 ? code_byte<2>(code[x]) : code_byte<3>(code[x]));
            const int p0 = 2 * (y & 1);
            const uint32_t cb = reinterpret_cast<const uint32_t(&)[4]>(cw[x])[y];
            float v0 = __uint_as_float(cb << 16) + fmaf(magic(at, p0, one), dc[x].s[p0], dc[x].m[p0]);
            float v1 = __uint_as_float(cb & 0xffff0000u) +
                       fmaf(magic(at, p0 + 1, one), dc[x].s[p0 + 1], dc[x].m[p0 + 1]);
            if (comp) {
              v0 = fmaf(corr[2 * x], cs[x], v0);
              v1 = fmaf(corr[2 * x + 1], cs[x], v1);
            }
            out[x][4 * hf + y] = pack_bf16(v0, v1);
          }
        }
      }
      uint16_t* dst = (kv ? V : K) + c * KCH + 16 * wa;
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (live[x]) store32(dst + (size_t)(g + 8 * x) * D, out[x]);
    }
  }
}

template <int D, bool TAB, int RK>
__global__ void __launch_bounds__(32 * NW_UNPACK, 1) unpack_kernel(const __grid_constant__ UnpackArgs A) {
  extern __shared__ __align__(128) uint8_t smem[];
  const Fields F = fields_of<D, NW_UNPACK, RK>(A.Dm);
  const int64_t x0 = blockIdx.x * A.total / gridDim.x, x1 = (blockIdx.x + 1) * A.total / gridDim.x;
  for (int64_t x = x0; x < x1;) {
    const int hr = (int)(x / A.nt);  // head of this call
    const int64_t head0 = (int64_t)hr * A.nt;
    const int64_t end = head0 + A.nt < x1 ? head0 + A.nt : x1;
    const int64_t tend = (end - head0) * KT < A.T ? (end - head0) * KT : A.T;
    uint16_t* const K = A.K + (size_t)hr * A.T * D;
    uint16_t* const V = A.V + (size_t)hr * A.T * D;
    walk<D, NW_UNPACK, TAB, RK>(
        A.Dm, A.v, F, smem, A.h0 + hr, (x - head0) * KT, tend,
        [&](const uint8_t* pk, int lo, int hi, int64_t t, const uint16_t* gk, const uint16_t* gv) {
          const size_t o = (size_t)t * KT * D;
          unpack16<D, TAB, RK>(A, F, pk, smem, gk, gv, lo, hi, K + o, V + o);
        });
    __syncthreads();  // the tables are done with
    x = end;
  }
}

constexpr uint32_t kMostSmem = 227 * 1024;

template <int D, bool TAB, int RK>
cudaError_t launch_rows(const RowsArgs& a, int grid, cudaStream_t s) {
  uint32_t tab = TAB ? 2u * a.Dm.C * D * 2 : 0u;
  if (tab < merge_bytes<D>()) tab = merge_bytes<D>();
  const uint32_t bytes = fields_of<D, NW_ROWS, RK>(a.Dm).tab + tab;
  if (bytes > kMostSmem) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(rows_kernel<D, TAB, RK>, allowed, (int)kMostSmem);
  if (e != cudaSuccess) return e;
  rows_kernel<D, TAB, RK><<<(unsigned)grid, 32 * NW_ROWS, bytes, s>>>(a);
  return cudaGetLastError();
}

template <int D, bool TAB, int RK>
cudaError_t launch_unpack(const UnpackArgs& a, int grid, cudaStream_t s) {
  const uint32_t tab = TAB ? 2u * a.Dm.C * D * 2 : 0u;
  const uint32_t bytes = fields_of<D, NW_UNPACK, RK>(a.Dm).tab + tab;
  if (bytes > kMostSmem) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(unpack_kernel<D, TAB, RK>, allowed, (int)kMostSmem);
  if (e != cudaSuccess) return e;
  unpack_kernel<D, TAB, RK><<<(unsigned)grid, 32 * NW_UNPACK, bytes, s>>>(a);
  return cudaGetLastError();
}

// Both centroid tables of a head fit in shared memory beside the rest.
bool tables_fit(const Dims& D) { return (int64_t)D.C * D.d <= 32768; }

// f.run<D, TAB, RK>() of the variant that serves a cache; tab: with staged tables (FIT64:
// always so at head 64, where up to 512 centroids fit).
template <bool FIT64, class F>
cudaError_t variant(const Dims& D, bool tab, F f) {
  const bool deep = D.r > 8;
  if (D.d == 128) {
    if (tab) return deep ? f.template run<128, true, 16>() : f.template run<128, true, 8>();
    return deep ? f.template run<128, false, 16>() : f.template run<128, false, 8>();
  }
  if constexpr (!FIT64)
    if (!tab) return deep ? f.template run<64, false, 16>() : f.template run<64, false, 8>();
  return deep ? f.template run<64, true, 16>() : f.template run<64, true, 8>();
}

struct RunRows {
  const RowsArgs& a;
  int grid;
  cudaStream_t s;
  template <int D, bool TAB, int RK>
  cudaError_t run() { return launch_rows<D, TAB, RK>(a, grid, s); }
};
struct RunUnpack {
  const UnpackArgs& a;
  int grid;
  cudaStream_t s;
  template <int D, bool TAB, int RK>
  cudaError_t run() { return launch_unpack<D, TAB, RK>(a, grid, s); }
};

}  // namespace

cudaError_t launch_unpack(const Dims& D, const CacheView& v, int64_t T, int h0, int heads, uint16_t* K,
                               uint16_t* V, int sms, cudaStream_t s) {
  UnpackArgs a = {};
  a.Dm = D;
  a.v = v;
  a.T = T;
  a.nt = (T + KT - 1) / KT;
  a.total = a.nt * heads;
  a.h0 = h0;
  a.K = K;
  a.V = V;
  const int64_t most = (a.total + NW_UNPACK - 1) / NW_UNPACK;  // CTAs with a tile for every warp
  const int grid = (int)(most < sms ? most : sms);
  // Staging both tables of a head pays from about 32 keys per centroid in a block's run
  // on: at 256 centroids 40 x 9360 tokens (2530 keys per block) take 7 us less without,
  // 40 x 37440 (10118 keys) 9 us more; at 16 centroids 40 x 9360 3 us more.  (The
  // attention of few rows takes as long or longer without at every length.)
  const bool tab = tables_fit(D) && a.total * KT >= (int64_t)grid * 32 * D.C;
  return variant<false>(D, tab, RunUnpack{a, grid, s});
}

// Rows of one product, and a history that gives every warp four tiles.  Otherwise the
// history is unpacked and attended to as bf16: at 40 heads x 37440 tokens 16 rows take
// 248 us here and 357 us there, and a second row tile, decoding all again, would take
// 463 us; 8 rows over 4 x 37440 tokens (5.3 tiles a warp) 54 and 69 us, over 40 x 3120
// (4.4) 55 and 56, over 12 x 7919 (3.3) 48 and 46, one row there 46 and 40.  (64 partials
// leave one key head 62 CTAs: 8 rows over 115200 tokens 66 us here, 63 unpacked; two heads
// of 57600 tokens, on 124 CTAs, 50 and 57.)
bool rows_supported(const Dims& D, int64_t T, int64_t rows, int sms) {
  return rows <= 16 && (T + KT - 1) / KT * D.H >= 4 * (int64_t)NW_ROWS * sms;
}

RowsPlan rows_plan(const Dims& D, int64_t T, int sms, int most) {
  RowsPlan p;
  const int64_t nt = (T + KT - 1) / KT, total = nt * D.H;
  // a head's nt tiles meet at most nt grid / total + 2 CTAs' runs
  int64_t grid = sms < total ? sms : total;
  if (grid / D.H + 2 > most) grid = (int64_t)D.H * (most - 2 > 0 ? most - 2 : 1);
  if (grid > total) grid = total;
  p.grid = (int)grid;
  p.slots = (int)(grid / D.H + 2);
  return p;
}

cudaError_t launch_rows(const Dims& D, const CacheView& v, int64_t T, const uint16_t* Q, int64_t ldq,
                        int64_t nq, int Hq, float scale_log2, const RowsPlan& plan, float* ws_o,
                        float* ws_l, cudaStream_t s) {
  RowsArgs a = {};
  a.Dm = D;
  a.v = v;
  a.T = T;
  a.Q = Q;
  a.ldq = ldq;
  a.g = Hq / D.H;
  a.rows = (int)(nq * a.g);
  a.Hq = Hq;
  a.scale_log2 = scale_log2;
  a.ws_o = ws_o;
  a.ws_l = ws_l;
  a.nq = nq;
  a.nslot = plan.slots;
  a.nt = (T + KT - 1) / KT;
  a.total = a.nt * D.H;
  return variant<true>(D, tables_fit(D), RunRows{a, plan.grid, s});
}

}  // namespace qwm
