// rope.cu -- per-head RMS norm with the position rotation in one pass
// (qwm_norm_rope), and the same on the way into a paged bf16 cache
// (qwm_paged_append).
//
//   y = x rsqrt(mean_j x_j^2 + eps) w,
//   (a, b) -> gain (a cos t - b sin t, a sin t + b cos t),  t = pos freq.
//
// Bound by memory: every element is read once and written once, 4 bytes per
// element; but at 6.5 TB/s an SM has only about 6 operations for each, so the
// arithmetic is kept short: with pairs (a, b), weights and turn fold into four
// factors per pair and token, a' = inv (a A1 - b A2), b' = inv (b B1 + a B2), two
// pairs to an instruction.  A lane holds whole pairs: four of an interleaved
// 16-byte chunk, or the eight of the two partner chunks of the half layout (with
// the partner in another lane, shuffles and a second unpacking made the
// operations the bound).  The mean is a butterfly over a row's lanes.
//
// One warp serves a token's query or key heads (or, with few tokens, a slice of
// them) by itself: no barrier ties its latencies (the angles, a page's place) to
// other warps', and its next rows are on the way while it works on these.
// Measured: the 480p frame (1560 x 80 heads x 128, normed and rotated) 10.9 us,
// 5.9 TB/s; 9361 x 48 heads in the half layout, half of each head, 44.0 us, 5.2 TB/s; a
// paged append of 5072 x 12 heads 17.1 us, 3.6 TB/s.  A block per token took 18.3, 102 and 44 us.
//
// Angles are formed in fp64 and reduced to half turns in (-1, 1] before the fp32
// sincospif: in fp32 a position near 10^6 would be off by 0.06 rad.  A lane computes one or
// two pairs for all of the warp's rows, through shared memory, which keeps the
// fp64 work at 1 / heads of the elements.
#include <math.h>

#include "around.cuh"
#include "tc.cuh"

namespace qwm {

namespace {

// Set when an offset or page number of a device array lay outside its buffer.
__device__ int g_index_fault;

constexpr int32_t kRopeMagic = 0x51575250;  // "QWRP"
constexpr int NT = 128;      // threads per block; 5 blocks per SM (102 registers) did better than 4 or 6
constexpr int UNROLL = 4;    // 16-byte pieces per lane and step; as many again are on the way

struct Side {
  const uint16_t* x;  // rows, ld apart
  const uint16_t* w;  // [D] norm weights or null
  uint16_t* out;      // rows, ldo apart; paged: the pool
  int64_t ld, ldo;
  int heads;
};

struct RopeArgs {
  Side s[2];  // queries and keys; paged: keys and values
  const int32_t* pos;
  int64_t ldpos, n;
  int64_t units;         // (token, side, slice) of all
  int slices0, slices;   // of the first side, of both, per token
  int per_slice;         // heads
  int pairs, end0, end1;  // pairs; first pair behind axis 0 and axis 1
  float gain, eps;
  // paged
  const int32_t *table, *cu, *start;
  int64_t n_seq, n_pages;
  int width, shift;  // table columns; log2 of the page size
  double freq[QWM_ROPE_MAX_PAIRS];
};

enum { ROT_NONE = 0, ROT_HALF = 1, ROT_INTER = 2 };

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// The pairs of a lane, a and b, from its NC chunks of 8 channels and back: pair e
// is channels 2e, 2e + 1 of the chunk (NC = 1), or channel e of both (NC = 2).
template <int NC>
__device__ __forceinline__ void pairs_of(const uint4 (&v)[NC], float (&a)[4 * NC], float (&b)[4 * NC]) {
  const uint32_t(&x)[4] = reinterpret_cast<const uint32_t(&)[4]>(v[0]);
  const uint32_t(&y)[4] = reinterpret_cast<const uint32_t(&)[4]>(v[NC - 1]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (NC == 1) {
      a[i] = low(x[i]);
      b[i] = high(x[i]);
    } else {
      a[2 * i] = low(x[i]);
      a[2 * i + 1] = high(x[i]);
      b[2 * i] = low(y[i]);
      b[2 * i + 1] = high(y[i]);
    }
  }
}
template <int NC>
__device__ __forceinline__ void chunks_of(const float (&a)[4 * NC], const float (&b)[4 * NC], uint4 (&v)[NC]) {
  if constexpr (NC == 1) {
    v[0] = make_uint4(pack2(a[0], b[0]), pack2(a[1], b[1]), pack2(a[2], b[2]), pack2(a[3], b[3]));
  } else {
    v[0] = make_uint4(pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(a[4], a[5]), pack2(a[6], a[7]));
    v[1] = make_uint4(pack2(b[0], b[1]), pack2(b[2], b[3]), pack2(b[4], b[5]), pack2(b[6], b[7]));
  }
}

// Cosine and sine of pos * freq.  k = the nearest whole number of turns; the
// two-part 2 pi keeps the remainder's error near that of the product itself
// (2^-53 of the angle: below 3e-7 rad for every int32 position).
__device__ __forceinline__ float2 turn(int pos, double freq, float gain) {
  const double a = (double)pos * freq;
  const double k = rint(a * 0.15915494309189535);
  double r = fma(k, -6.283185307179586, a);
  r = fma(k, -2.4492935982947064e-16, r);
  float s, c;
  sincospif((float)(r * 0.3183098861837907), &s, &c);
  return make_float2(c * gain, s * gain);
}

// Place of row t's position in the pools, as an element offset of head 0, or -1:
// a row of no sequence, or a page outside the pool or the table.  One warp; the
// sequence is the last that begins at or before t, found by 32 probes at a time; where
// its positions start comes with the probes, a load's latency earlier.
__device__ __forceinline__ int64_t place_of(const RopeArgs& A, int64_t t, int D) {
  const int lane = threadIdx.x & 31;
  int64_t lo = -1, hi = A.n_seq + 1;  // cu[lo] <= t < cu[hi]
  int begin = 0, start = 0;           // of lo
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 31) / 32, x = lo + (lane + 1) * step;
    const int c = x < hi ? __ldg(A.cu + x) : 0, s = x < A.n_seq ? __ldg(A.start + x) : 0;
    const unsigned below = __ballot_sync(0xffffffffu, x < hi && c <= t);
    const int n = below == 0xffffffffu ? 32 : __ffs(~below) - 1;  // the leading probes
    if (n > 0) {
      begin = __shfl_sync(0xffffffffu, c, n - 1);
      start = __shfl_sync(0xffffffffu, s, n - 1);
    }
    const int64_t up = lo + (n + 1) * step;
    lo += n * step;
    hi = up < hi ? up : hi;
  }
  if (lo < 0 || lo >= A.n_seq) return -1;
  const int64_t p = (int64_t)start + (t - begin);
  const int64_t col = p >> A.shift;
  int64_t page = -1;
  if (p >= 0 && col < A.width) page = __ldg(A.table + lo * A.width + col);
  if (page < 0 || page >= A.n_pages) {
    if (lane == 0) atomicExch(&g_index_fault, 1);
    return -1;
  }
  return (((page * A.s[0].heads) << A.shift) + (p & ((1 << A.shift) - 1))) * D;
}

// FULL: every channel is rotated.  Otherwise the lanes behind rot_dim skip the sums over a
// pair, for a NaN or an infinity there is its own channel's alone; the test takes 4 % of a
// 480p frame's time where no lane needs it (11.6 against 11.1 us; the two forms behind one
// branch, 12.0).
template <int D, int ROT, bool FULL, bool PAGED>
__global__ void __launch_bounds__(NT, 5) norm_rope_kernel(const __grid_constant__ RopeArgs A) {
  using namespace tc;
  constexpr int NC = ROT == ROT_HALF ? 2 : 1;  // chunks of a lane
  constexpr int NP = 4 * NC;                   // pairs of a lane
  constexpr int L = D / (8 * NC);              // lanes per row
  constexpr int ROWS = 32 / L;                 // rows per warp at once
  constexpr int U = UNROLL / NC;               // of them in a step
  constexpr int STEP = ROWS * U;
  __shared__ float2 cs_all[ROT ? NT / 32 * QWM_ROPE_MAX_PAIRS : 1];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (NT / 32) + warp;
  if (unit >= A.units) return;
  const int64_t t = (uint32_t)unit / (uint32_t)A.slices;  // (the host keeps units in 32 bits)
  const int slice = (int)(unit - t * A.slices), side = slice >= A.slices0;
  const Side& S = A.s[side];
  const int h0 = (side ? slice - A.slices0 : slice) * A.per_slice;
  const int h1 = h0 + A.per_slice < S.heads ? h0 + A.per_slice : S.heads;
  const bool values = PAGED && side == 1;  // copied as they are
  const int c = lane % L, row = lane / L;
  // the lane's chunks: c; or partners c and c + half / 8, and neighbours behind them
  const int nr = ROT == ROT_HALF ? A.pairs / 8 : 0;
  int at[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) at[i] = 8 * (NC == 1 ? c : c < nr ? c + i * nr : 2 * c + i);
  const uint16_t* const xt = S.x + t * S.ld;
  auto load = [&](uint4 (&v)[U][NC], int h) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        v[u][i] = make_uint4(0, 0, 0, 0);
        if (h + row + u * ROWS < h1)
          v[u][i] = *reinterpret_cast<const uint4*>(xt + (int64_t)(h + row + u * ROWS) * D + at[i]);
      }
  };
  uint4 now[U][NC];
  load(now, h0);
  float2* cs = cs_all + (ROT ? warp * QWM_ROPE_MAX_PAIRS : 0);
  if (ROT && !values) {
    for (int i = lane; i < A.pairs; i += 32) {
      const int axis = (i >= A.end0) + (i >= A.end1);
      cs[i] = turn(__ldg(A.pos + axis * A.ldpos + t), A.freq[i], A.gain);
    }
  }
  int64_t place = 0;
  if (PAGED) {
    place = place_of(A, t, D);
    if (place < 0) return;
  }
  __syncwarp();

  const bool turns = ROT && NP * c < A.pairs;
  const int64_t oh = PAGED ? (int64_t)D << A.shift : D;  // from head to head
  const bool norm = !values && S.w != nullptr;
  uint64_t a1[NP / 2], a2[NP / 2], b1[NP / 2], b2[NP / 2];  // the factors, by twos
  if (!values && (ROT || norm)) {
    float wa[NP], wb[NP];
#pragma unroll
    for (int e = 0; e < NP; ++e) wa[e] = wb[e] = 1.0f;
    if (norm) {
      uint4 w[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(S.w + at[i]));
      pairs_of<NC>(w, wa, wb);
    }
#pragma unroll
    for (int e = 0; e < NP; e += 2) {
      float2 x = make_float2(1.0f, 0.0f), y = x;
      if (turns) {
        x = cs[NP * c + e];
        y = cs[NP * c + e + 1];
      }
      a1[e / 2] = f2pack(wa[e] * x.x, wa[e + 1] * y.x);
      a2[e / 2] = f2pack(-wb[e] * x.y, -wb[e + 1] * y.y);
      b1[e / 2] = f2pack(wb[e] * x.x, wb[e + 1] * y.x);
      b2[e / 2] = f2pack(wa[e] * x.y, wa[e + 1] * y.y);
    }
  }
  uint16_t* const ot = S.out + (PAGED ? place : t * S.ldo);
  for (int h = h0; h < h1; h += STEP) {
    uint4 next[U][NC];
    load(next, h + STEP);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!values && (ROT || norm)) {
        float a[NP], b[NP];
        pairs_of<NC>(now[u], a, b);
        uint64_t inv2 = f2pack(1.0f, 1.0f);
        if (norm) {
          uint64_t sq = 0;
#pragma unroll
          for (int e = 0; e < NP; e += 2) {
            const uint64_t x = f2pack(a[e], a[e + 1]), y = f2pack(b[e], b[e + 1]);
            sq = ffma2(x, x, sq);
            sq = ffma2(y, y, sq);
          }
          float s0, s1;
          f2unpack(sq, s0, s1);
          float ss = s0 + s1;
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, L);
          const float inv = rsqrtf(ss * (1.0f / D) + A.eps);
          inv2 = f2pack(inv, inv);
        }
#pragma unroll
        for (int e = 0; e < NP; e += 2) {
          const uint64_t x = f2pack(a[e], a[e + 1]), y = f2pack(b[e], b[e + 1]);
          uint64_t p = fmul2(x, a1[e / 2]), q = fmul2(y, b1[e / 2]);
          if (ROT && (FULL || turns)) {  // a channel behind rot_dim takes nothing from its neighbour
            p = ffma2(y, a2[e / 2], p);
            q = ffma2(x, b2[e / 2], q);
          }
          if (norm) {
            p = fmul2(p, inv2);
            q = fmul2(q, inv2);
          }
          f2unpack(p, a[e], a[e + 1]);
          f2unpack(q, b[e], b[e + 1]);
        }
        chunks_of<NC>(a, b, now[u]);
      }
      if (h + row + u * ROWS < h1) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
          *reinterpret_cast<uint4*>(ot + (h + row + u * ROWS) * oh + at[i]) = now[u][i];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NC; ++i) now[u][i] = next[u][i];
  }
}

// A warp per token and side keeps the angles' share small; with few tokens the
// heads are sliced, down to a step of rows, until 16 warps per SM have work.
constexpr int MOST_HEADS = 64;  // per slice

template <int D>
void set_units(RopeArgs& a) {
  const int step = 32 / (D / 8) * UNROLL;
  for (int per = MOST_HEADS;; per /= 2) {
    a.per_slice = per;
    a.slices0 = (a.s[0].heads + per - 1) / per;
    a.slices = a.slices0 + (a.s[1].heads + per - 1) / per;
    a.units = a.n * a.slices;
    if (per <= step || a.units >= 148 * 16) return;
  }
}

template <int D, bool PAGED>
cudaError_t launch(RopeArgs& a, int rot, cudaStream_t s) {
  set_units<D>(a);
  const unsigned grid = (unsigned)((a.units + NT / 32 - 1) / (NT / 32));
  const bool full = 2 * a.pairs == D;
  if (rot == ROT_NONE) norm_rope_kernel<D, ROT_NONE, false, PAGED><<<grid, NT, 0, s>>>(a);
  else if (rot == ROT_HALF && full) norm_rope_kernel<D, ROT_HALF, true, PAGED><<<grid, NT, 0, s>>>(a);
  else if (rot == ROT_HALF) norm_rope_kernel<D, ROT_HALF, false, PAGED><<<grid, NT, 0, s>>>(a);
  else if (full) norm_rope_kernel<D, ROT_INTER, true, PAGED><<<grid, NT, 0, s>>>(a);
  else norm_rope_kernel<D, ROT_INTER, false, PAGED><<<grid, NT, 0, s>>>(a);
  return cudaGetLastError();
}

// The kernel counts units in 31 bits (with that many rows a slice is as long as it gets).
bool units_ok(int64_t n, int32_t heads0, int32_t heads1) {
  const int64_t slices = (heads0 + MOST_HEADS - 1) / MOST_HEADS + (heads1 + MOST_HEADS - 1) / MOST_HEADS;
  return n <= (int64_t(1) << 31) - 1 && n * slices <= (int64_t(1) << 31) - 1;
}

bool rope_ok(const qwm_rope* r, int32_t head_dim) {
  if (r->magic != kRopeMagic || r->head_dim != head_dim) return false;
  return true;
}

bool row_ok(int64_t ld, int32_t heads, int32_t head_dim) {
  return ld >= (int64_t)heads * head_dim && ld % 8 == 0;
}

void set_rope(RopeArgs& a, const qwm_rope* r) {
  a.pairs = r->rot_dim / 2;
  a.end0 = r->axis_dim[0] / 2;
  a.end1 = r->n_axes > 1 ? a.end0 + r->axis_dim[1] / 2 : a.pairs;
  a.gain = (float)r->gain;
  for (int i = 0; i < a.pairs; ++i) a.freq[i] = r->freq[i];
}

int rot_of(const qwm_rope* r) {
  return !r ? ROT_NONE : r->layout == QWM_ROPE_HALF ? ROT_HALF : ROT_INTER;
}

}  // namespace

int read_and_clear_append_fault() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_index_fault, sizeof(int)) != cudaSuccess) return -1;
  if (v) cudaMemcpyToSymbol(g_index_fault, &z, sizeof(int));
  return v;
}

}  // namespace qwm

using namespace qwm;

extern "C" qwm_status qwm_rope_init(qwm_rope* r, int32_t head_dim, int32_t rot_dim, int32_t layout,
                                    double theta, int32_t n_axes, const int32_t* axis_dim,
                                    int32_t scaling, double factor, double orig_len,
                                    double beta_fast, double beta_slow) {
  if (!r || (head_dim != 64 && head_dim != 128)) return QWM_ERR_INVALID_ARG;
  if (rot_dim < 16 || rot_dim > head_dim || rot_dim % 16) return QWM_ERR_INVALID_ARG;
  if (layout != QWM_ROPE_HALF && layout != QWM_ROPE_INTERLEAVED) return QWM_ERR_INVALID_ARG;
  if (n_axes < 1 || n_axes > QWM_ROPE_MAX_AXES || (!axis_dim && n_axes != 1))
    return QWM_ERR_INVALID_ARG;
  if (scaling < QWM_ROPE_SCALE_NONE || scaling > QWM_ROPE_SCALE_PARTS) return QWM_ERR_INVALID_ARG;
  // written so that a NaN fails each test
  if (!(theta > 1.0) || !isfinite(theta) || !(factor >= 1.0) || !isfinite(factor))
    return QWM_ERR_INVALID_ARG;
  if (scaling == QWM_ROPE_SCALE_PARTS &&
      (!(orig_len > 0.0) || !isfinite(orig_len) || !(beta_slow >= 0.0) ||
       !(beta_fast > beta_slow) || !isfinite(beta_fast)))
    return QWM_ERR_INVALID_ARG;
  int64_t sum = 0;
  for (int a = 0; a < n_axes; ++a) {
    const int32_t dim = axis_dim ? axis_dim[a] : rot_dim;
    if (dim < 2 || dim % 2 || (scaling == QWM_ROPE_SCALE_NTK && dim < 4))
      return QWM_ERR_INVALID_ARG;
    sum += dim;
  }
  if (sum != rot_dim) return QWM_ERR_INVALID_ARG;
  const double pi = 3.14159265358979323846;
  qwm_rope t = {};
  t.head_dim = head_dim;
  t.rot_dim = rot_dim;
  t.layout = layout;
  t.n_axes = n_axes;
  t.gain = scaling == QWM_ROPE_SCALE_PARTS ? 0.1 * log(factor) + 1.0 : 1.0;
  int pair = 0;
  for (int a = 0; a < n_axes; ++a) {
    const int32_t dim = axis_dim ? axis_dim[a] : rot_dim;
    t.axis_dim[a] = dim;
    const double base = scaling == QWM_ROPE_SCALE_NTK
                            ? theta * pow(factor, (double)dim / (double)(dim - 2))
                            : theta;
    for (int i = 0; i < dim / 2; ++i, ++pair) {
      double f = pow(base, -2.0 * i / dim);
      if (scaling == QWM_ROPE_SCALE_LINEAR) f /= factor;
      if (scaling == QWM_ROPE_SCALE_PARTS) {
        double keep = (orig_len * f / (2.0 * pi) - beta_slow) / (beta_fast - beta_slow);
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        f = keep * f + (1.0 - keep) * f / factor;
      }
      t.freq[pair] = f;
    }
  }
  t.magic = kRopeMagic;
  *r = t;
  return QWM_OK;
}

extern "C" qwm_status qwm_norm_rope(const qwm_rope* rope, int32_t head_dim, int64_t n,
                                    const void* Q, int64_t ldq, int32_t heads_q, const void* w_q,
                                    void* Q_out, int64_t ldqo, const void* K, int64_t ldk,
                                    int32_t heads_k, const void* w_k, void* K_out, int64_t ldko,
                                    const int32_t* pos, int64_t ldpos, float eps, void* stream) {
  if ((head_dim != 64 && head_dim != 128) || n < 0 || !(eps >= 0.0f) || heads_q < 0 || heads_k < 0 ||
      heads_q > 65536 || heads_k > 65536 || !units_ok(n, heads_q, heads_k))
    return QWM_ERR_INVALID_ARG;
  if (rope && (!rope_ok(rope, head_dim) || (n > 0 && !pos) || ldpos < n)) return QWM_ERR_INVALID_ARG;
  RopeArgs a = {};
  const void* x[2] = {Q, K};
  const void* w[2] = {w_q, w_k};
  void* o[2] = {Q_out, K_out};
  const int64_t ld[2] = {ldq, ldk}, ldo[2] = {ldqo, ldko};
  const int32_t heads[2] = {heads_q, heads_k};
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    if (n > 0 && (!x[i] || !o[i])) return QWM_ERR_INVALID_ARG;
    if (!row_ok(ld[i], heads[i], head_dim) || !row_ok(ldo[i], heads[i], head_dim))
      return QWM_ERR_INVALID_ARG;
    if (x[i] == o[i] && ld[i] != ldo[i]) return QWM_ERR_INVALID_ARG;
    if (!aligned_to(x[i], 16) || !aligned_to(o[i], 16) || !aligned_to(w[i], 16))
      return QWM_ERR_ALIGNMENT;
    a.s[i] = Side{(const uint16_t*)x[i], (const uint16_t*)w[i], (uint16_t*)o[i], ld[i], ldo[i],
                  heads[i]};
  }
  if (rope && !aligned_to(pos, 4)) return QWM_ERR_ALIGNMENT;
  if (n == 0 || heads_q + heads_k == 0) return QWM_OK;
  a.pos = pos;
  a.ldpos = ldpos;
  a.n = n;
  a.eps = eps;
  if (rope) set_rope(a, rope);
  const cudaError_t e = head_dim == 128 ? launch<128, false>(a, rot_of(rope), (cudaStream_t)stream)
                                        : launch<64, false>(a, rot_of(rope), (cudaStream_t)stream);
  return e == cudaSuccess ? QWM_OK : QWM_ERR_CUDA;
}

extern "C" qwm_status qwm_paged_append(const qwm_pages* p, const int32_t* table, int64_t n_seq,
                                       int32_t table_width, const int32_t* cu,
                                       const int32_t* start, const void* K, int64_t ldk,
                                       const void* V, int64_t ldv, int64_t n, const qwm_rope* rope,
                                       const int32_t* pos, int64_t ldpos, const void* w_k,
                                       float eps, void* stream) {
  if (!pages_ok(p) || n < 0 || !units_ok(n, p->heads, p->heads) || n_seq < 1 || n_seq > (1 << 24) ||
      table_width < 1 || !table || !cu || !start || !(eps >= 0.0f) || (n > 0 && (!K || !V)))
    return QWM_ERR_INVALID_ARG;
  if (rope && (!rope_ok(rope, p->head_dim) || (n > 0 && !pos) || ldpos < n))
    return QWM_ERR_INVALID_ARG;
  if (!row_ok(ldk, p->heads, p->head_dim) || !row_ok(ldv, p->heads, p->head_dim))
    return QWM_ERR_INVALID_ARG;
  if (!aligned_to(p->K, 16) || !aligned_to(p->V, 16) || !aligned_to(K, 16) || !aligned_to(V, 16) ||
      !aligned_to(w_k, 16) || !aligned_to(table, 4) || !aligned_to(cu, 4) ||
      !aligned_to(start, 4) || (rope && !aligned_to(pos, 4)))
    return QWM_ERR_ALIGNMENT;
  if (n == 0) return QWM_OK;
  RopeArgs a = {};
  a.s[0] = Side{(const uint16_t*)K, (const uint16_t*)w_k, (uint16_t*)p->K, ldk, 0, p->heads};
  a.s[1] = Side{(const uint16_t*)V, nullptr, (uint16_t*)p->V, ldv, 0, p->heads};
  a.pos = pos;
  a.ldpos = ldpos;
  a.n = n;
  a.eps = eps;
  a.table = table;
  a.cu = cu;
  a.start = start;
  a.n_seq = n_seq;
  a.n_pages = p->n_pages;
  a.width = table_width;
  a.shift = page_shift(p);
  if (rope) set_rope(a, rope);
  const cudaError_t e = p->head_dim == 128
                            ? launch<128, true>(a, rot_of(rope), (cudaStream_t)stream)
                            : launch<64, true>(a, rot_of(rope), (cudaStream_t)stream);
  return e == cudaSuccess ? QWM_OK : QWM_ERR_CUDA;
}
