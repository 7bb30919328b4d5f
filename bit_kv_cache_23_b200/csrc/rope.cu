// rope.cu -- per-head RMS norm with the position rotation in one pass
// (qwm_norm_rope), and the same on the way into a paged bf16 cache
// (qwm_paged_append).
//
//   y = x rsqrt(mean_j x_j^2 + eps) w,
//   (a, b) -> gain (a cos t - b sin t, a sin t + b cos t),  t = pos freq.
//
// Bound by memory: every element is read once and written once, 4 bytes per
// element and about 10 fp32 operations.  A head's row lies in D/8 adjacent
// lanes, 16 bytes each, so the mean is a butterfly over those lanes and the
// partner of a half-layout pair comes from another lane by shuffles; a lane
// keeps its channels' cosines, sines and weights in registers over the rows of
// one token.
//
// Angles are formed in fp64 and reduced to (-pi, pi] before the fp32 sincosf:
// in fp32 a position near 10^6 would be off by 0.06 rad.  One thread computes
// each (token, pair) once for all heads of the block's tokens, through shared
// memory, which keeps the fp64 work at 1 / heads of the elements.
#include <math.h>

#include "around.cuh"

namespace qwm {

namespace {

// Set when an offset or page number of a device array lay outside its buffer.
__device__ int g_index_fault;

constexpr int32_t kRopeMagic = 0x51575250;  // "QWRP"
constexpr int NT = 256;                     // threads per block
constexpr int UNROLL = 4;                   // rows in flight per lane
constexpr int MAX_TB = 4;                   // tokens per block at most

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
  int tb;    // tokens per block: 1, 2 or 4
  int pairs, end0, end1;  // pairs; first pair behind axis 0 and axis 1
  float gain, eps;
  // paged
  const int32_t *table, *cu, *start;
  int64_t n_seq, n_pages;
  int width, shift;  // table columns; log2 of the page size
  double freq[QWM_ROPE_MAX_PAIRS];
};

enum { ROT_NONE = 0, ROT_HALF = 1, ROT_INTER = 2 };

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
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
  sincosf((float)r, &s, &c);
  return make_float2(c * gain, s * gain);
}

// Place of position p of sequence b in a pool, as an element offset of head 0,
// or -1 for a page outside the pool or the table.
__device__ __forceinline__ int64_t place_of(const RopeArgs& A, int64_t t, int D) {
  // the last sequence that begins at or before row t
  int64_t lo = 0, hi = A.n_seq;  // cu[lo] <= t < cu[hi], where rows are owned
  if (t >= A.cu[A.n_seq] || t < A.cu[0]) return -1;  // behind the last sequence: left alone
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (A.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int64_t p = (int64_t)A.start[lo] + (t - A.cu[lo]);
  const int64_t col = p >> A.shift;
  int64_t page = -1;
  if (p >= 0 && col < A.width) page = A.table[lo * A.width + col];
  if (page < 0 || page >= A.n_pages) {
    atomicExch(&g_index_fault, 1);
    return -1;
  }
  return (((page * A.s[0].heads) << A.shift) + (p & ((1 << A.shift) - 1))) * D;
}

template <int D, int ROT, bool PAGED>
__global__ void __launch_bounds__(NT) norm_rope_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int L = D / 8;        // lanes per row
  constexpr int GROUPS = NT / L;  // rows per block and step
  __shared__ float2 cs[ROT ? MAX_TB * QWM_ROPE_MAX_PAIRS : 1];
  __shared__ int64_t place[MAX_TB];
  const int64_t t0 = (int64_t)blockIdx.x * A.tb;
  if (ROT) {
    for (int e = threadIdx.x; e < A.tb * A.pairs; e += NT) {
      const int tl = e / A.pairs, i = e - tl * A.pairs;
      if (t0 + tl < A.n) {
        const int axis = (i >= A.end0) + (i >= A.end1);
        cs[tl * QWM_ROPE_MAX_PAIRS + i] =
            turn(__ldg(A.pos + axis * A.ldpos + t0 + tl), A.freq[i], A.gain);
      }
    }
  }
  if (PAGED && threadIdx.x < A.tb)
    place[threadIdx.x] = t0 + threadIdx.x < A.n ? place_of(A, t0 + threadIdx.x, D) : -1;
  __syncthreads();

  const int c = threadIdx.x % L;  // this lane's 8 channels: 8c .. 8c+7
  const int grp = threadIdx.x / L;
  const int tl = grp % A.tb, h0 = grp / A.tb, step = GROUPS / A.tb;
  const int64_t t = t0 + tl;
  const bool live = t < A.n && (!PAGED || place[tl] >= 0);
  const int half = A.pairs / 8;  // chunks of half the rotated channels
  const bool turns = ROT && c < 2 * half;
  // the lane that holds the partners of a half-layout pair
  const int partner = ROT == ROT_HALF && turns ? (c < half ? c + half : c - half) : c;
  float co[ROT == ROT_HALF ? 8 : 4], si[ROT == ROT_HALF ? 8 : 4];
  if (ROT) {
    constexpr int NP = ROT == ROT_HALF ? 8 : 4;
    const int first = ROT == ROT_HALF ? 8 * (c < half ? c : c - half) : 4 * c;
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      float2 v = make_float2(1.0f, 0.0f);
      if (turns && live) v = cs[tl * QWM_ROPE_MAX_PAIRS + first + e];
      co[e] = v.x;
      si[e] = (ROT == ROT_HALF && c < half) ? -v.y : v.y;
    }
  }
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const Side& S = A.s[side];
    const bool values = PAGED && side == 1;  // copied as they are
    float w[8], pw[ROT == ROT_HALF ? 8 : 1];
    const bool norm = S.w != nullptr;
    if (norm) {
      unpack8(__ldg(reinterpret_cast<const uint4*>(S.w) + c), w);
      if constexpr (ROT == ROT_HALF)
        unpack8(__ldg(reinterpret_cast<const uint4*>(S.w) + partner), pw);
    }
    const uint16_t* xt = S.x + t * S.ld + 8 * c;
    uint16_t* ot = S.out + 8 * c + (PAGED ? place[tl] : t * S.ldo);
    const int64_t oh = PAGED ? (int64_t)D << A.shift : D;  // from head to head
    for (int hb = h0; hb - h0 < S.heads; hb += step * UNROLL) {
      uint4 raw[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int h = hb + u * step;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (live && h < S.heads) raw[u] = *reinterpret_cast<const uint4*>(xt + (int64_t)h * D);
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int h = hb + u * step;
        uint4 res = raw[u];
        if (!values && (ROT || norm)) {
          float v[8];
          unpack8(raw[u], v);
          float inv = 1.0f;
          if (norm) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, L);
            inv = rsqrtf(ss * (1.0f / D) + A.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * inv * w[e];
          }
          if constexpr (ROT == ROT_HALF) {
            uint4 pr;
            pr.x = __shfl_sync(0xffffffffu, raw[u].x, partner, L);
            pr.y = __shfl_sync(0xffffffffu, raw[u].y, partner, L);
            pr.z = __shfl_sync(0xffffffffu, raw[u].z, partner, L);
            pr.w = __shfl_sync(0xffffffffu, raw[u].w, partner, L);
            float p[8];
            unpack8(pr, p);
            if (norm) {
#pragma unroll
              for (int e = 0; e < 8; ++e) p[e] = p[e] * inv * pw[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = turns ? fmaf(p[e], si[e], v[e] * co[e]) : v[e];
          }
          if constexpr (ROT == ROT_INTER) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = v[2 * e], b = v[2 * e + 1];
              v[2 * e] = turns ? fmaf(-b, si[e], a * co[e]) : a;
              v[2 * e + 1] = turns ? fmaf(a, si[e], b * co[e]) : b;
            }
          }
          res = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]),
                           pack2(v[6], v[7]));
        }
        if (live && h < S.heads) *reinterpret_cast<uint4*>(ot + h * oh) = res;
      }
    }
  }
}

template <int D, bool PAGED>
cudaError_t launch(const RopeArgs& a, int rot, cudaStream_t s) {
  const unsigned grid = (unsigned)((a.n + a.tb - 1) / a.tb);
  if (rot == ROT_NONE) norm_rope_kernel<D, ROT_NONE, PAGED><<<grid, NT, 0, s>>>(a);
  else if (rot == ROT_HALF) norm_rope_kernel<D, ROT_HALF, PAGED><<<grid, NT, 0, s>>>(a);
  else norm_rope_kernel<D, ROT_INTER, PAGED><<<grid, NT, 0, s>>>(a);
  return cudaGetLastError();
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

// Tokens per block: with few tokens one each, so that they spread over the SMs;
// with many, four, so that one fp64 angle per thread covers the block's pairs.
int tokens_per_block(int64_t n) { return n >= 4096 ? 4 : n >= 1024 ? 2 : 1; }

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
  if ((head_dim != 64 && head_dim != 128) || n < 0 || n > (int64_t(1) << 31) - 1 || !(eps >= 0.0f) ||
      heads_q < 0 || heads_k < 0 || heads_q > 65536 || heads_k > 65536)
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
  a.tb = tokens_per_block(n);
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
  if (!pages_ok(p) || n < 0 || n > (int64_t(1) << 31) - 1 || n_seq < 1 || n_seq > (1 << 24) ||
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
  a.tb = tokens_per_block(n);
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
