// attention_rows.cu -- attention of few query rows per head (single tokens of a
// few branches) over the packed cache, decoded straight into the operands of
// register-level matrix products: nothing but the packed fields crosses HBM.
//
// Bound by the decoding, not by memory: at 40 heads x 37440 tokens x 128 channels
// the packed fields are 162 MB (25 us), while every element takes about four
// instructions to rebuild.  So the layout serves the decoder.  A warp takes 16
// keys at a time; in the products' operand layout (lane = 4 g + c) the channels
// are permuted such that a lane owns a quarter head of keys g and g + 8 of K'
// (whole INT2 groups: two code words, one or two parameter words per key) and
// D / 8 channels of keys 2c, 2c+1, 2c+8, 2c+9 of V', and each decoded pair goes
// from the conversion into its product without passing through shared memory.
//
//   K'  = bf16((c + mn + code sc) + cs sum_i U_i c8_i).  The compensation is a
//         product too: c8 is exact in bf16, and U, split into three bf16 parts
//         (24 bits), stays in registers as the B operand while its version lasts.
//   S   = Q K'^T, P = 2^(scale log2e S - m), O += P V': m16n8k16, rows = queries.
//
// Each CTA takes an equal run of (head, 128-key chunk) positions, whatever the
// number of heads, and gives one partial per head it touches; its eight warps
// share a chunk (16 keys each), keep a running maximum, sum and O of their own
// and meet at the end of a head.  The head's centroid tables lie in shared
// memory when both fit (C D <= 32768), tokens of another table version, and
// larger tables, are read through the cache.  The packed fields of the chunks
// ahead are copied into a ring; the warp that is last to leave a stage refills it.
#include <math.h>

#include "around.cuh"
#include "dequant_pairs.cuh"
#include "tc.cuh"

namespace qwm {
namespace {
using namespace tc;

__device__ int g_rows_timeout;

constexpr int CH = 128;       // keys per chunk
constexpr int NW = 8;         // decoding warps
constexpr int NTHREADS = 32 * NW;  // 255 registers per thread
constexpr int NSTAGE = 3;
constexpr int MAX_R = 8;      // PSAC rank served here
constexpr float TAU = 8.0f;   // a row's reference moves when its maximum grew by more (log2)

struct RowsArgs {
  Dims Dm;
  CacheView v;
  int64_t T;
  const uint16_t* Q;
  int64_t ldq, rows;   // rows per head: tokens x query heads of a key head
  int Hq, g;
  float scale_log2;
  float *ws_o, *ws_l;  // [slot][token][Hq][D], [slot][token][Hq]
  int64_t nq;
  int nslot;           // slots of a head
  int64_t nc, total;   // chunks per head, in all
  int tables;          // both centroid tables in shared memory
};

// Stage: the packed fields of 128 keys.
template <int D>
struct RLay {
  static constexpr uint32_t KC = 0, VC = KC + CH * D / 4, KP = VC + CH * D / 4,
                            VP = KP + CH * (D / 16) * 4, CO = VP + CH * (D / 16) * 4,
                            CS = CO + CH * MAX_R, KI = CS + CH * 2, VI = KI + CH * 2,
                            TV = VI + CH * 2, CV = TV + CH * 2, STAGE = CV + CH * 2;
  static constexpr uint32_t OFF_BAR = 0;                       // copies landed; warps done
  static constexpr uint32_t OFF_ML = 2 * NSTAGE * 8 + 16;      // [warp][16] m, l
  static constexpr uint32_t OFF_Q = (OFF_ML + 2 * NW * 16 * 4 + 127) / 128 * 128;  // [16][D] bf16
  static constexpr uint32_t OFF_ST = OFF_Q + 16 * D * 2;
  static constexpr uint32_t OFF_TAB = OFF_ST + NSTAGE * STAGE;  // tables, or the warps' O
  static constexpr uint32_t MERGE = NW * 16 * D * 4;
};
static_assert(RLay<128>::OFF_TAB + 2 * 32768 * 2 <= 227 * 1024, "shared memory");

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(uint64_t v) {
  float a, b;
  f2unpack(v, a, b);
  return pack_bf16(a, b);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), bf16; and with 8 in place of 16.
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

__device__ __forceinline__ void timeout_flag() { atomicExch(&g_rows_timeout, 1); }

// The CTA whose run holds position x.
__device__ __forceinline__ int64_t cta_of(const RowsArgs& A, int64_t x) {
  return ((x + 1) * gridDim.x - 1) / A.total;
}

// Copy the fields of the chunk at position x into stage s (one thread).
template <int D>
__device__ __forceinline__ void fill_stage(const RowsArgs& A, uint8_t* smem, uint64_t* full,
                                           volatile int* issued, int64_t x, int s) {
  using L = RLay<D>;
  const Dims& Dm = A.Dm;
  const int ng = Dm.ng, r = Dm.r, ib = Dm.idx_bytes;
  const int h = (int)(x / A.nc);
  const int64_t t0 = (x - (int64_t)h * A.nc) * CH;
  const PackedHead p = packed_head(A.v, Dm, h);
  const uint32_t st = smem_u32(smem) + L::OFF_ST + s * L::STAGE;
  uint64_t* bar = &full[s];
  issued[s] = issued[s] + 1;
  mbar_arrive_expect_tx(bar, 2 * (CH * D / 4) + 2 * CH * ng * 4 + (r > 0 ? CH * r + CH * 2 : 0) +
                                 2 * CH * 2 + 2 * CH * ib);
  bulk_g2s(st + L::KC, p.k_codes + t0 * (D / 4), CH * D / 4, bar);
  bulk_g2s(st + L::VC, p.v_codes + t0 * (D / 4), CH * D / 4, bar);
  bulk_g2s(st + L::KP, p.k_params + t0 * ng * 2, CH * ng * 4, bar);
  bulk_g2s(st + L::VP, p.v_params + t0 * ng * 2, CH * ng * 4, bar);
  if (r > 0) {
    bulk_g2s(st + L::CO, p.k_coef + t0 * r, CH * r, bar);
    bulk_g2s(st + L::CS, p.k_cscale + t0, CH * 2, bar);
  }
  bulk_g2s(st + L::TV, A.v.tokver + t0, CH * 2, bar);
  bulk_g2s(st + L::CV, A.v.centver + t0, CH * 2, bar);
  bulk_g2s(st + L::KI, (const uint8_t*)p.k_idx + t0 * ib, CH * ib, bar);
  bulk_g2s(st + L::VI, (const uint8_t*)p.v_idx + t0 * ib, CH * ib, bar);
}

// What a decoding warp keeps while it works on one head.
template <int D>
struct State {
  float o[D / 8][4];      // O: n-tile j holds channels g' D/8 + j; rows g, g + 8
  float m0, m1, l0, l1;   // reference and (this lane's part of the) sum of rows g, g + 8
  uint32_t u[D / 8][3];   // U of version `uver`: high, middle and low bf16 parts
  int uver;
};

// U of head h, version ver, as B operands: n-tile j's column n is channel
// (n / 2) D/4 + 2j + n % 2, so that a lane's accumulators are its own channels.
template <int D>
__device__ __forceinline__ void load_basis(const RowsArgs& A, int h, int ver, State<D>& st) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int r = A.Dm.r;
  const float* U = basis_of(A.v, A.Dm, ver, h);
#pragma unroll
  for (int j = 0; j < D / 8; ++j) {
    const int ch = (g >> 1) * (D / 4) + 2 * j + (g & 1);
    float x[2];
    uint32_t part[3];
#pragma unroll
    for (int e = 0; e < 2; ++e) x[e] = 2 * c + e < r ? __ldg(U + (size_t)ch * r + 2 * c + e) : 0.0f;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      part[k] = pack_bf16(x[0], x[1]);
      x[0] -= __uint_as_float(part[k] << 16);  // exact: the rounding's remainder
      x[1] -= __uint_as_float(part[k] & 0xffff0000u);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) st.u[j][k] = part[k];
  }
  st.uver = ver;
}

__device__ __forceinline__ uint32_t i8_pair_bf16(uint32_t two) {
  return pack_bf16(i8_to_f32((int8_t)(two & 0xff)), i8_to_f32((int8_t)(two >> 8)));
}

// One warp: the 16 keys at k0 of the staged chunk (nval of the chunk's keys are
// cached; the fields of the others are not used).
template <int D>
__device__ __forceinline__ void keys16(const RowsArgs& A, const uint8_t* pk, const uint8_t* smem,
                                       int h, int k0, int nval, int tabver, State<D>& st) {
  using L = RLay<D>;
  constexpr int KCH = D / 4;  // a lane's K channels
  constexpr int VCH = D / 8;  // a lane's V channels
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const Dims& Dm = A.Dm;
  const int G = Dm.G, ng = Dm.ng, r = Dm.r, ib = Dm.idx_bytes;
  const uint16_t* tv = reinterpret_cast<const uint16_t*>(pk + L::TV);
  const uint16_t* cv = reinterpret_cast<const uint16_t*>(pk + L::CV);
  const uint8_t* tab = smem + L::OFF_TAB;
  const size_t hoff = (size_t)h * Dm.C * D;
  const size_t vstride = cent_slot_elems(Dm);
  // row of a centroid table: staged, or in memory
  auto centroid = [&](const uint16_t* table, uint32_t staged, uint32_t fields, int k, bool live) {
    const int idx = !live ? 0
                    : ib == 1 ? (int)pk[fields + k]
                              : (int)reinterpret_cast<const uint16_t*>(pk + fields)[k];
    const int ver = live ? cv[k] : tabver;
    return ver == tabver && A.tables
               ? reinterpret_cast<const uint4*>(tab + staged + (uint32_t)idx * (D * 2))
               : reinterpret_cast<const uint4*>(table + ver * vstride + hoff + (size_t)idx * D);
  };

  // ---- K' of keys g and g + 8, and S
  float s[2][4];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[x][e] = 0.0f;
  {
    const uint4* cp[2];
    uint32_t code[2][KCH / 16];
    GroupConst gc[2][KCH / 16];
    uint64_t cs2[2];
    uint32_t a[2] = {0, 0};
    bool same = true;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int k = k0 + g + 8 * x;
      const bool live = k < nval;
      cp[x] = centroid(A.v.cent_k, 0, L::KI, k, live) + c * (KCH / 8);
#pragma unroll
      for (int w = 0; w < KCH / 16; ++w) {
        code[x][w] = reinterpret_cast<const uint32_t*>(pk + L::KC)[k * (D / 16) + c * (KCH / 16) + w];
        gc[x][w] = group_const(
            reinterpret_cast<const uint32_t*>(pk + L::KP)[k * ng + (c * KCH + 16 * w) / G]);
      }
      cs2[x] = 0;
      if (r > 0) {
        const float cs = live ? half_bits_to_f32(reinterpret_cast<const uint16_t*>(pk + L::CS)[k]) : 0.0f;
        cs2[x] = f2pack(cs, cs);
        uint32_t two = 0;
        if (2 * c < r) two = pk[L::CO + k * r + 2 * c];
        if (2 * c + 1 < r) two |= (uint32_t)pk[L::CO + k * r + 2 * c + 1] << 8;
        a[x] = i8_pair_bf16(two);
        same &= !live || tv[k] == tv[k0];
      }
    }
    same = __all_sync(0xffffffffu, same);
    if (r > 0 && same && st.uver != tv[k0]) load_basis<D>(A, h, tv[k0], st);
    const uint4* qs = reinterpret_cast<const uint4*>(smem + L::OFF_Q);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {  // a lane's channels 4 ks .. 4 ks + 3
      uint32_t b[2][2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int j = 2 * ks + y;  // channels 2j, 2j + 1
        float corr[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (r > 0) {
          if (same) {
            mma16(corr, a[0], a[1], a[0], a[1], st.u[j][0], st.u[j][1]);
            mma8(corr, a[0], a[1], st.u[j][2]);
          } else {  // keys of several basis versions: once per refresh
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int k = k0 + g + 8 * x;
              if (k >= nval) continue;
              const float* U = basis_of(A.v, Dm, tv[k], h) + (size_t)(c * KCH + 2 * j) * r;
              for (int q = 0; q < r; ++q) {
                const float f = (float)(int8_t)pk[L::CO + k * r + q];
                corr[2 * x] = fmaf(__ldg(U + q), f, corr[2 * x]);
                corr[2 * x + 1] = fmaf(__ldg(U + r + q), f, corr[2 * x + 1]);
              }
            }
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          // code pair j of word j / 8: byte (j % 8) / 2, positions 2 (j % 2), + 1
          const uint32_t w = code[x][j / 8];
          const int byte = (j % 8) / 2, pos = 2 * (j % 2);
          const uint32_t at = byte == 0 ? w << 15 : byte == 1 ? w << 7 : byte == 2 ? w >> 1 : w >> 9;
          const GroupConst& q = gc[x][j / 8];
          const uint64_t mm = f2pack(magic_code(at, pos), magic_code(at, pos + 1));
          const uint32_t cw = reinterpret_cast<const uint32_t*>(cp[x])[j];
          uint64_t v = ffma2(mm, pos == 0 ? q.s01 : q.s23, pos == 0 ? q.m01 : q.m23);
          v = fadd2(f2pack(__uint_as_float(cw << 16), __uint_as_float(cw & 0xffff0000u)), v);
          if (r > 0) v = ffma2(f2pack(corr[2 * x], corr[2 * x + 1]), cs2[x], v);
          b[x][y] = pack_bf16(v);
        }
      }
      // Q rows g and g + 8, the same four channels
      const uint4 q = qs[ks * 32 + lane];
      mma16(s[0], q.x, q.z, q.y, q.w, b[0][0], b[0][1]);
      mma16(s[1], q.x, q.z, q.y, q.w, b[1][0], b[1][1]);
    }
  }

  // ---- softmax: this lane's keys 2c, 2c + 1 (s[0]) and 8 + 2c, 9 + 2c (s[1])
  uint32_t p[4];
  {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool live = k0 + 8 * x + 2 * c + e < nval;
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
      // (some key of the 16 is cached, so the new references are finite)
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

  // ---- V' of keys 2c, 2c + 1 (pair 0) and 2c + 8, 2c + 9 (pair 1), and O
  {
    const uint4* cp[4];
    uint32_t code[4];
    uint64_t S[2][4], M[2][4];  // [pair][position in the code byte]
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      GroupConst q[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = k0 + 2 * c + 8 * x + e;
        const bool live = k < nval;
        cp[2 * x + e] = centroid(A.v.cent_v, Dm.C * D * 2, L::VI, k, live) + g * (VCH / 8);
        const uint8_t* cd = pk + L::VC + k * (D / 4) + g * (VCH / 4);
        code[2 * x + e] = VCH == 16 ? *reinterpret_cast<const uint32_t*>(cd)
                                    : *reinterpret_cast<const uint16_t*>(cd);
        // a key that is not cached: finite (its weight is 0)
        q[e] = group_const(live ? reinterpret_cast<const uint32_t*>(pk + L::VP)[k * ng + g * VCH / G] : 0u);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float a0, a1, b0, b1;
        f2unpack(e ? q[0].s23 : q[0].s01, a0, a1);
        f2unpack(e ? q[1].s23 : q[1].s01, b0, b1);
        S[x][2 * e] = f2pack(a0, b0);
        S[x][2 * e + 1] = f2pack(a1, b1);
        f2unpack(e ? q[0].m23 : q[0].m01, a0, a1);
        f2unpack(e ? q[1].m23 : q[1].m01, b0, b1);
        M[x][2 * e] = f2pack(a0, b0);
        M[x][2 * e + 1] = f2pack(a1, b1);
      }
    }
#pragma unroll
    for (int j8 = 0; j8 < VCH / 8; ++j8) {
      uint4 cw[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) cw[k] = cp[k][j8];
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        const int j = 8 * j8 + jj, byte = j / 4, pos = j % 4;
        uint32_t b[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float mm[2], cc[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t w = code[2 * x + e];
            const uint32_t at = byte == 0 ? w << 15 : byte == 1 ? w << 7 : byte == 2 ? w >> 1 : w >> 9;
            mm[e] = magic_code(at, pos);
            const uint32_t q = reinterpret_cast<const uint32_t(&)[4]>(cw[2 * x + e])[jj / 2];
            cc[e] = __uint_as_float(jj & 1 ? q & 0xffff0000u : q << 16);
          }
          b[x] = pack_bf16(fadd2(f2pack(cc[0], cc[1]), ffma2(f2pack(mm[0], mm[1]), S[x][pos], M[x][pos])));
        }
        mma16(st.o[j], p[0], p[1], p[2], p[3], b[0], b[1]);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1) rows_kernel(const __grid_constant__ RowsArgs A) {
  using L = RLay<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  int* done = reinterpret_cast<int*>(full + NSTAGE);  // warps that have left a stage
  volatile int* issued = done + NSTAGE;               // copies into it
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t x0 = blockIdx.x * A.total / gridDim.x, x1 = (blockIdx.x + 1) * A.total / gridDim.x;
  const int64_t r0 = (int64_t)blockIdx.y * 16;  // first row of this row tile
  if (threadIdx.x == 0) {
    for (int i = 0; i < NSTAGE; ++i) {
      mbar_init(&full[i], 1);
      done[i] = 0;
      issued[i] = 0;
    }
    fence_mbar_init();
    fence_proxy_async_smem();
    for (int i = 0; i < NSTAGE && x0 + i < x1; ++i) fill_stage<D>(A, smem, full, issued, x0 + i, i);
  }
  __syncthreads();
  const Dims& Dm = A.Dm;
  State<D> st;
  bool ok = true;
  int n = 0;
  for (int64_t x = x0; x < x1;) {
    const int h = (int)(x / A.nc);
    const int64_t head_end = (int64_t)(h + 1) * A.nc;
    const int64_t end = head_end < x1 ? head_end : x1;
    // ---- this head's Q rows (operand order: four channels of rows g and g + 8 per lane)
    __syncthreads();  // the last head's tables, O and Q are done with
    for (int e = threadIdx.x; e < (D / 16) * 32; e += 32 * NW) {
      const int ks = e >> 5, gg = (e & 31) >> 2, cc = e & 3;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int64_t r = r0 + gg + 8 * y;
        uint2 q = make_uint2(0, 0);
        if (r < A.rows) {
          const int64_t tok = r / A.g;
          q = __ldg(reinterpret_cast<const uint2*>(
              A.Q + tok * A.ldq + ((int64_t)h * A.g + (r - tok * A.g)) * D + cc * (D / 4) + 4 * ks));
        }
        *reinterpret_cast<uint2*>(smem + L::OFF_Q + e * 16 + 8 * y) = q;
      }
    }
    int tabver = -1;
    st.uver = -1;
    st.m0 = st.m1 = -INFINITY;
    st.l0 = st.l1 = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[j][e] = 0.0f;
    for (; x < end; ++x, ++n) {
      const int64_t t0 = (x - (int64_t)h * A.nc) * CH;
      const int nval = (int)(A.T - t0 < CH ? A.T - t0 : CH);
      const int s = n % NSTAGE;
      // after a timeout the warp still meets the others at the barriers
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[s], (n / NSTAGE) & 1));
      const uint8_t* pk = smem + L::OFF_ST + s * L::STAGE;
      // table version of the chunk's first key, the same for every warp
      const int ver = ok ? reinterpret_cast<const uint16_t*>(pk + L::CV)[0] : A.v.centver[t0];
      if (ver != tabver) {
        __syncthreads();
        if (A.tables) {
          const size_t off = (size_t)ver * cent_slot_elems(Dm) + (size_t)h * Dm.C * D;
          const uint4* sk = reinterpret_cast<const uint4*>(A.v.cent_k + off);
          const uint4* sv = reinterpret_cast<const uint4*>(A.v.cent_v + off);
          uint4* d = reinterpret_cast<uint4*>(smem + L::OFF_TAB);
          const int words = Dm.C * D / 8;
          for (int e = threadIdx.x; e < words; e += 32 * NW) {
            d[e] = __ldg(sk + e);
            d[words + e] = __ldg(sv + e);
          }
        }
        tabver = ver;
        __syncthreads();
      }
      if (ok && 16 * warp < nval) keys16<D>(A, pk, smem, h, 16 * warp, nval, tabver, st);
      __syncwarp();
      if (lane == 0) {
        __threadfence_block();
        if (atomicAdd(&done[s], 1) == NW - 1) {  // (the others' reads are before their add)
          done[s] = 0;
          __threadfence_block();
          if (ok && x + NSTAGE < x1) fill_stage<D>(A, smem, full, issued, x + NSTAGE, s);
        }
      }
    }
    // ---- the warps' results: maxima and sums, then O over the tables' place
    float* ml = reinterpret_cast<float*>(smem + L::OFF_ML);
    float* ow = reinterpret_cast<float*>(smem + L::OFF_TAB);
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
    const int slot = (int)(blockIdx.x - cta_of(A, (int64_t)h * A.nc));
    for (int e = threadIdx.x; e < 16 * D; e += 32 * NW) {
      const int row = e / D, ch = e % D;
      const int64_t r = r0 + row;
      if (r >= A.rows) break;  // rows ascend
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
      const int64_t tok = r / A.g;
      const int64_t out = tok * A.Hq + (int64_t)h * A.g + (r - tok * A.g);
      A.ws_o[((size_t)slot * A.nq * A.Hq + out) * D + ch] = o / l;
      if (ch == 0) {
        A.ws_l[(size_t)slot * A.nq * A.Hq + out] = (top + log2f(l)) * 0.6931471805599453f;
        // the head's last run says which slots stay empty
        if (end == head_end)
          for (int k = slot + 1; k < A.nslot; ++k) A.ws_l[(size_t)k * A.nq * A.Hq + out] = -INFINITY;
      }
    }
  }
  if (!ok && lane == 0) {
    timeout_flag();
    // copies that were issued land before the CTA exits
    for (int i = 0; i < NSTAGE; ++i)
      if (issued[i] > 0) mbar_wait(&full[i], (issued[i] - 1) & 1);
  }
}

template <int D>
cudaError_t launch_rows(const RowsArgs& a, int grid, int tiles, cudaStream_t s) {
  using L = RLay<D>;
  uint32_t tab = a.tables ? 2u * a.Dm.C * D * 2 : 0u;
  if (tab < L::MERGE) tab = L::MERGE;
  const int bytes = (int)(L::OFF_TAB + tab);
  cudaError_t e = cudaFuncSetAttribute(rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  rows_kernel<D><<<dim3((unsigned)grid, (unsigned)tiles), NTHREADS, bytes, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

// At most this many rows per head run here: up to two 16-row tiles, which decode
// the history once each.
bool rows_supported(const Dims& D, int64_t rows) { return D.r <= MAX_R && rows <= 32; }

RowsPlan rows_plan(const Dims& D, int64_t T, int sms, int most) {
  RowsPlan p;
  const int64_t nc = (T + CH - 1) / CH, total = nc * D.H;
  // a head's run of nc chunks meets at most nc grid / total + 2 CTAs' runs
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
  a.rows = nq * a.g;
  a.Hq = Hq;
  a.scale_log2 = scale_log2;
  a.ws_o = ws_o;
  a.ws_l = ws_l;
  a.nq = nq;
  a.nslot = plan.slots;
  a.nc = (T + CH - 1) / CH;
  a.total = a.nc * D.H;
  a.tables = (int64_t)D.C * D.d <= 32768;
  const int tiles = (int)((a.rows + 15) / 16);
  return D.d == 128 ? launch_rows<128>(a, plan.grid, tiles, s) : launch_rows<64>(a, plan.grid, tiles, s);
}

int read_and_clear_rows_timeout() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_rows_timeout, sizeof(int)) != cudaSuccess) return -1;
  if (v) cudaMemcpyToSymbol(g_rows_timeout, &z, sizeof(int));
  return v;
}

}  // namespace qwm
