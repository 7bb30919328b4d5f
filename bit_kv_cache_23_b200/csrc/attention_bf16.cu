// attention_bf16.cu -- attention over bf16 keys on the sm_100a tensor cores
// (tcgen05.mma; S, P and O live in TMEM), for queries whose keys come from two
// sources in turn: keys that all sequences share, then each sequence's own.
//   qwm_attention_shared  shared: the packed history, unpacked once per head
//                         into the workspace; own: pages.
//   qwm_cross_attention   shared: none; own: rows of an encoder's states.
//
//   S = Q K^T,  m = running row maximum,  P = 2^(scale log2e S - m),
//   l = sum P,  O = sum P V,  out = O / l,  lse = ln 2 (m + log2 l).
//
// One CTA serves up to 128 query rows of one key head (the query heads that share
// the key head are rows too) over a range of 64-key tiles; nothing but Q, K, V and
// the result crosses HBM.  With too few row blocks to fill the GPU the key range is
// split; each range gives a normalized fp32 partial and its log-sum-exp, which a
// last kernel merges.
//
// 192 threads: warps 0-3 softmax (one row per thread), warp 4 the loader, warp 5
// the issuing thread.  Two score buffers in TMEM let Q K^T of the next tiles run
// while the softmax works on this one.  Two CTAs share an SM: one's products run
// while the other has the exponential unit, and one's beginning and end hide
// behind the other's tiles.  (One CTA of 256 rows, with each K and V tile read
// once for two such groups, took 8 to 18 % longer up to 2048 keys, as long at 4096 and
// 5 % less at 8192: the groups fall into step, both waiting for products and then both
// for the exponential unit.  That was with one lane issuing the products, which bounded
// every form then; it was not measured again with the warp that issues them now.)
//
// Bound, with tiles of 64 keys, by the tensor core's reading of shared memory, and by the
// power limit: a 128 x 64 tile's products take 643 cycles, of which S takes 386 (a product of 64
// columns reads 6 KB in 48 cycles for 32 cycles of arithmetic; 128 columns would
// take 64, but two such buffers beside O do not fit in half of TMEM), and an SM with
// two CTAs needs 720 cycles per tile.  1560 rows x 40 heads over 8192 keys: 243 to 247
// us, 1060 to 1080 TFLOP/s, at 1.6 GHz; 592 even row blocks 1170 TFLOP/s.
//
// K and V tiles go through one ring of TMA boxes in the 128-byte-swizzled layout
// that the MMA descriptors read (one box per 64 channels and, for pages, per
// page).  What lies behind a sequence's end never meets a product: boxes beyond
// a tensor arrive as zeros, and the loader overwrites the V rows behind the end
// of the last tile with zeros (scores of hidden keys are replaced, so K rows may
// hold anything).
//
// Every mbarrier wait is bounded (about 1 s) and reported by qwm_device_status.
#include <cuda.h>
#include <math.h>

#include "around.cuh"
#include "tc.cuh"

namespace qwm {
namespace {
using namespace tc;

__device__ int g_flash_timeout;
__device__ int g_flash_fault;  // a length, offset or page number was clamped

constexpr int KT = 64;           // keys per tile
constexpr int QT = 128;          // query rows per Q tile (TMEM lanes)

constexpr int W_LOAD = 4, W_MMA = 5, NTHREADS = 192;
constexpr uint32_t COLS = 256;   // TMEM: S, S, O

template <int D>
struct Lay {
  static constexpr uint32_t Q_TILE = QT * D * 2;  // [D / 64 column blocks][128 rows][128 B]
  static constexpr uint32_t ENT = KT * D * 2;     // one K or V tile, [D / 64][64 rows][128 B]
  static constexpr uint32_t OFF_K = Q_TILE, OFF_V = OFF_K + 2 * ENT;  // two tiles of each
  static constexpr uint32_t OFF_BAR = OFF_V + 2 * ENT;
  // Tile t uses places and barriers t & 1.  Few barriers, for each commit costs the
  // issuing thread time: S is also what frees K's place, P V what frees V's.
  static constexpr int B_K = 0,           // loader -> MMA
                       B_V = B_K + 2,
                       B_S = B_V + 2,     // commit of Q K^T -> softmax, loader
                       B_P = B_S + 2,     // softmax -> MMA
                       B_PV = B_P + 2,    // commit of P V -> softmax, loader
                       B_Q = B_PV + 2,    // Q is in shared memory
                       B_DONE = B_Q + 1, // drain before exit
                       B_RAG = B_DONE + 1,  // a ragged V tile has landed -> loader
                       NBAR = B_RAG + 1;
  static constexpr uint32_t SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
};
static_assert(Lay<128>::SMEM <= 113 * 1024 && Lay<64>::SMEM <= 113 * 1024, "two CTAs per SM");

constexpr int kMostKeys = (1 << 30);  // of a sequence, rows alike: sums of both stay in 31 bits

enum { OWN_NONE = 0, OWN_ROWS = 1, OWN_PAGES = 2 };

struct FlashArgs {
  const uint16_t* Q;
  int64_t ldq, nq;
  int Hq, g;           // query heads; query heads per key head
  const int32_t* cu;   // [n_seq + 1], or null: one sequence of all rows
  int64_t max_q;       // rows of a sequence at most
  // keys that every sequence sees first (maps: channel, key, head of the pass)
  int64_t len0;
  // keys of each sequence (maps: channel, key head, row; pages: channel, head and
  // place in the page, page)
  int own;
  int64_t n_kv;                 // rows
  const int32_t *kv_start, *kv_len, *table;
  int64_t max_kv, n_pages;
  int width, shift;             // pages
  int causal;
  float scale_log2;
  uint16_t* O;
  float* lse;          // or null
  int head0;           // first key head of the pass
  int qblocks, nsplit;
  int part0;           // first partial of this launch; -1: no partials
  float *ws_o, *ws_l;  // [partial][nq][Hq][D], [partial][nq][Hq]
  int qtma;            // Q rows come through the map (g divides 128)
  CUtensorMap q, k0, v0, k1, v1;
};

// What one CTA does: rows r0 .. r0 + nr - 1 of sequence b (a row is a token
// and one of the g query heads of key head h), key tiles j0 .. j0 + n - 1.
struct Work {
  int64_t tok0;    // first token row of the sequence
  int nb;          // its tokens
  int r0;
  int nr;          // rows of this CTA
  int h;
  int len1;        // own keys that are read (at most max_kv)
  int len;         // own keys of the sequence
  int start1;      // first own row (OWN_ROWS)
  int b;
  int nt0;         // tiles of the shared keys
  int j0, n, part;
  // row r's token
  __device__ __forceinline__ int token(const FlashArgs& A, int r) const {
    return A.g == 1 ? r : r / A.g;
  }
  // own keys that row r sees (causal)
  __device__ __forceinline__ int seen(const FlashArgs& A, int r) const {
    const int x = len - nb + token(A, r) + 1;
    return x < 0 ? 0 : x > len1 ? len1 : x;
  }
};

__device__ __forceinline__ bool work_of(const FlashArgs& A, Work& w) {
  const int split = A.nsplit == 1 ? 0 : blockIdx.x / A.qblocks, qb = blockIdx.x - split * A.qblocks;
  w.h = A.head0 + blockIdx.y;
  w.b = blockIdx.z;
  w.part = A.part0 + split;
  // all loads at once (each takes about 400 cycles)
  const bool seqs = A.cu != nullptr, keys = A.own != OWN_NONE, rows_own = A.own == OWN_ROWS;
  const int64_t c0 = seqs ? __ldg(A.cu + w.b) : 0, c1 = seqs ? __ldg(A.cu + w.b + 1) : A.nq;
  int64_t len = keys ? __ldg(A.kv_len + w.b) : 0;
  const int64_t start = rows_own ? __ldg(A.kv_start + w.b) : 0;
  bool fault = c0 < 0 || c1 < c0 || c1 > A.nq;
  w.tok0 = fault ? 0 : c0;
  w.nb = fault ? 0 : (int)(c1 - c0);
  // (the host refuses more than 2^31 - 1 rows, keys or pages' places)
  const int rows = (w.nb < A.max_q ? w.nb : (int)A.max_q) * A.g;
  w.r0 = qb * QT;
  w.len = w.len1 = 0;
  w.start1 = 0;
  if (keys) {
    int64_t room = A.own == OWN_PAGES ? (int64_t)A.width << A.shift : A.n_kv;
    if (rows_own) {
      fault |= start < 0 || start > A.n_kv;
      w.start1 = (int)(start < 0 ? 0 : start > A.n_kv ? A.n_kv : start);
      room -= w.start1;
    }
    fault |= len < 0 || len > room;
    len = len < 0 ? 0 : len > room ? room : len;
    w.len = (int)(len < kMostKeys ? len : kMostKeys);
    w.len1 = (int)(len < A.max_kv ? len : A.max_kv);
  }
  if (fault && threadIdx.x == 0) atomicExch(&g_flash_fault, 1);
  if (w.r0 >= rows) return false;
  w.nr = rows - w.r0 < QT ? rows - w.r0 : QT;
  const int seen = A.causal ? w.seen(A, w.r0 + w.nr - 1) : w.len1;  // own keys that the last row sees
  w.nt0 = (int)((A.len0 + KT - 1) / KT);
  const int nt = w.nt0 + (seen + KT - 1) / KT;
  w.j0 = 0;
  w.n = nt;
  if (A.nsplit > 1) {  // even ranges, the first ones a tile longer
    const int each = nt / A.nsplit, more = nt - each * A.nsplit;
    w.j0 = split * each + (split < more ? split : more);
    w.n = each + (split < more);
  }
  return true;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ void timeout_flag() { atomicExch(&g_flash_timeout, 1); }

__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  const bool w = mbar_wait(bar, parity);
  return __all_sync(0xffffffffu, w);
}

// ------------------------------------------------------------------ softmax role
// The exponent reference m_used moves only when the row maximum has grown by
// more than TAU (log2 units): P stays below 2^TAU, and O, which accumulates in
// TMEM, is rescaled in place on such moves only.
constexpr float TAU = 8.0f;

__device__ __forceinline__ float max64(const float (&s)[64]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < 64; e += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = fmax3(m[k], s[e + 2 * k], s[e + 2 * k + 1]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// P = 2^(sc S - m) of one row's 64 scores over the columns of S (bf16 pairs, keys
// 2i, 2i+1 in column i; rounded to nearest: 2^-8 relative per weight at most, l2
// sums the unrounded ones).
__device__ __forceinline__ void weights(float (&s)[64], uint64_t sc2, uint64_t nm2,
                                        uint64_t (&l2)[2], uint32_t ts) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 32 * c; e < 32 * c + 32; e += 2) {
      f2unpack(ffma2(f2pack(s[e], s[e + 1]), sc2, nm2), s[e], s[e + 1]);
      s[e] = ex2(s[e]);
      s[e + 1] = ex2(s[e + 1]);
    }
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      l2[0] = fadd2(l2[0], f2pack(s[32 * c + e], s[32 * c + e + 1]));
      l2[1] = fadd2(l2[1], f2pack(s[32 * c + e + 2], s[32 * c + e + 3]));
      pk[e / 2] = pack_bf16(s[32 * c + e], s[32 * c + e + 1]);
      pk[e / 2 + 1] = pack_bf16(s[32 * c + e + 2], s[32 * c + e + 3]);
    }
    tmem_st16u_nw(ts + 16 * c, pk);
  }
}

// Row r's place among O's rows.
__device__ __forceinline__ int64_t out_row(const FlashArgs& A, const Work& w, int r) {
  const int tok = w.token(A, r);
  return (w.tok0 + tok) * A.Hq + (w.h * A.g + (r - tok * A.g));
}

// 32 bytes, one sector, to a 32-byte aligned address.
__device__ __forceinline__ void store32(float* dst, const float* v, float f) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(v[0] * f), "f"(v[1] * f),
               "f"(v[2] * f), "f"(v[3] * f), "f"(v[4] * f), "f"(v[5] * f), "f"(v[6] * f), "f"(v[7] * f)
               : "memory");
}

// A warp's rows of O from TMEM, times each lane's `inv`, to this CTA's partial; row:
// the lane's row among O's.
template <int D>
__device__ __forceinline__ void store_part(const FlashArgs& A, const Work& w, bool valid, int64_t row, uint32_t to,
                                           float inv, float lse) {
  const size_t at = (size_t)w.part * A.nq * A.Hq + row;
  if (valid) A.ws_l[at] = lse;
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    float o[32];
    tmem_ld32(to + c * 32, o);
    if (!valid) continue;
#pragma unroll
    for (int k = 0; k < 32; k += 8) store32(A.ws_o + at * D + 32 * c + k, o + k, inv);
  }
}

// The same to O, through shared memory, where nothing is needed any more, so that a
// store covers whole rows (16-byte pieces exchanged by the row number keep the banks
// apart): four 720p frames of cross attention 210 us, 217 with each lane's pieces of
// its own row, 32 rows to a store.  (Of the fp32 partials those are whole sectors, and
// the way through shared memory took 1 % longer.)
template <int D>
__device__ __forceinline__ void store_rows(const FlashArgs& A, const Work& w, uint8_t* smem, bool valid,
                                           int64_t row, uint32_t to, float inv, float lse) {
  constexpr int RB = D * 2, UPR = RB / 16, RPI = 32 / UPR;  // bytes and pieces of a row; rows per store
  const int lane = threadIdx.x & 31;
  if (valid && A.lse) A.lse[row] = lse;
  uint8_t* const mine = smem + (threadIdx.x >> 5) * 32 * RB;
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    float o[32];
    tmem_ld32(to + c * 32, o);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<uint4*>(mine + lane * RB + (((4 * c + k) ^ (lane & 7)) << 4)) =
          make_uint4(pack_bf16(o[8 * k] * inv, o[8 * k + 1] * inv), pack_bf16(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                     pack_bf16(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                     pack_bf16(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
  }
  __syncwarp();
  const uint8_t* const src = mine + (lane / UPR) * RB;
  const int u = lane % UPR, left = w.nr - (int)(threadIdx.x & ~31u);  // rows of this warp and those behind
#pragma unroll 1
  for (int r0 = 0; r0 < 32 && r0 < left; r0 += 8 * RPI) {
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int rr = r0 + i * RPI;
      v[i] = *reinterpret_cast<const uint4*>(src + rr * RB + ((u ^ ((rr + lane / UPR) & 7)) << 4));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int rr = r0 + i * RPI + lane / UPR;
      const int64_t to_row = __shfl_sync(0xffffffffu, row, rr);
      if (rr < left) *reinterpret_cast<uint4*>(A.O + to_row * D + 8 * u) = v[i];
    }
  }
}

template <int D>
__device__ __forceinline__ void softmax_role(const FlashArgs& A, uint8_t* smem, uint64_t* bars,
                                             uint32_t tmem, const Work& w) {
  using L = Lay<D>;
  const int warp = threadIdx.x >> 5;
  if (!A.qtma) {  // Q rows into shared memory, zeros behind the last; eight loads in flight
    constexpr int C = D / 8, STEP = QT / C;
    const int c = threadIdx.x % C;
    for (int rr0 = threadIdx.x / C; rr0 < QT; rr0 += 8 * STEP) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int rr = rr0 + u * STEP;
        v[u] = make_uint4(0, 0, 0, 0);
        if (rr < w.nr) {
          const int r = w.r0 + rr, tok = w.token(A, r);
          v[u] = __ldg(reinterpret_cast<const uint4*>(A.Q + (w.tok0 + tok) * A.ldq +
                                                      (w.h * A.g + (r - tok * A.g)) * D + 8 * c));
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int rr = rr0 + u * STEP;
        if (rr < QT) *reinterpret_cast<uint4*>(smem + sw128_off(rr, c, QT)) = v[u];
      }
    }
    fence_proxy_async_smem();
    warp_arrive(&bars[L::B_Q]);
  }
  if (32 * warp >= w.nr) return;
  const int rr = threadIdx.x;  // row in the CTA and TMEM lane
  const bool valid = rr < w.nr;
  const int r = w.r0 + (valid ? rr : 0);
  const int seen = A.causal ? w.seen(A, r) : w.len1;  // own keys that this row sees
  // tiles with hidden keys: the shared keys' last, if not full, and own ones
  // from the first that some row of the warp does not see whole
  int cut0 = (int)(A.len0 % KT);
  if (cut0 == 0) cut0 = KT;
  const int whole = w.nt0 + __reduce_min_sync(0xffffffffu, seen) / KT;
  const uint32_t ts0 = tmem + ((uint32_t)(32 * warp) << 16), to = ts0 + 128;
  float m_used = -INFINITY;
  uint64_t l2[2] = {0, 0};  // running row sum, as pairs of partial sums
  const uint64_t sc2 = f2pack(A.scale_log2, A.scale_log2);
  bool ok = true;
  for (int i = 0; i < w.n; ++i) {
    const int j = w.j0 + i;
    const uint32_t ts = ts0 + 64 * (i & 1);
    if (!warp_wait(&bars[L::B_S + (i & 1)], (i >> 1) & 1)) { ok = false; break; }
    tc_fence_after();
    float s[64];
    tmem_ld64(ts, s);
    if ((j == w.nt0 - 1 && cut0 < KT) || j >= whole) {
      const int lim = j < w.nt0 ? cut0 : seen - (j - w.nt0) * KT;  // visible keys
#pragma unroll
      for (int e = 0; e < 64; ++e)
        if (e >= lim) s[e] = -INFINITY;
    }
    const float m_row = max64(s) * A.scale_log2;
    const bool need = m_row > m_used + TAU;  // (-inf + TAU = -inf: the first visible key)
    if (i == 0) {
      m_used = m_row;
    } else if (__any_sync(0xffffffffu, need)) {
      // O is at rest once the last product with P is complete (this tile's waits for P)
      if (!warp_wait(&bars[L::B_PV + ((i - 1) & 1)], ((i - 1) >> 1) & 1)) { ok = false; break; }
      tc_fence_after();
      const float f = need ? ex2(m_used - m_row) : 1.0f;
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {
        float o[16];
        tmem_ld16(to + c * 16, o);
        uint32_t ou[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) ou[e] = __float_as_uint(o[e] * f);
        tmem_st16u_nw(to + c * 16, ou);
      }
      l2[0] = ffma2(l2[0], f2pack(f, f), 0ull);
      l2[1] = ffma2(l2[1], f2pack(f, f), 0ull);
      if (need) m_used = m_row;
    }
    // a row that has seen no key yet: 2^(-inf - 0) = 0 rather than NaN
    const float mref = m_used == -INFINITY ? 0.0f : m_used;
    const uint64_t nm2 = f2pack(-mref, -mref);
    weights(s, sc2, nm2, l2, ts);
    tmem_wait_st();
    tc_fence_before();
    warp_arrive(&bars[L::B_P + (i & 1)]);
  }
  float la, lb;
  f2unpack(fadd2(l2[0], l2[1]), la, lb);
  const float l = la + lb;
  // (a row without keys; a NaN among the scores stays one)
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const float lse = l == 0.0f ? -INFINITY : (m_used + log2f(l)) * 0.6931471805599453f;
  const int64_t row = out_row(A, w, r);
  if (ok) ok = warp_wait(&bars[L::B_PV + ((w.n - 1) & 1)], ((w.n - 1) >> 1) & 1);
  if (!ok) {
    if ((threadIdx.x & 31) == 0) timeout_flag();
    return;
  }
  tc_fence_after();
  if (A.part0 >= 0) store_part<D>(A, w, valid, row, to, inv, lse);
  else store_rows<D>(A, w, smem, valid, row, to, inv, lse);
}

// ------------------------------------------------------------------ loader role
// All warps, from wherever they are: the barriers are set up, TMEM is there.
__device__ __forceinline__ void start_barrier() {
  asm volatile("barrier.sync 1, %0;" ::"n"(NTHREADS) : "memory");
}

// The boxes of K (v = 0) or V (v = 1) rows of key tile j to `dst`, ENT bytes
// in all; one thread.
template <int D>
__device__ __forceinline__ void issue_tile(const FlashArgs& A, const Work& w, int j, int v,
                                           uint32_t dst, uint64_t* bar) {
  constexpr uint32_t BLK = KT * 128;  // bytes of 64 channels of the tile
  if (j < w.nt0) {
    const CUtensorMap* m = v ? &A.v0 : &A.k0;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      tma_load_3d(dst + c * BLK, m, 64 * c, j * KT, w.h - A.head0, bar);
    return;
  }
  const CUtensorMap* m = v ? &A.v1 : &A.k1;
  const int k0 = (j - w.nt0) * KT;
  if (A.own == OWN_ROWS) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      tma_load_3d(dst + c * BLK, m, 64 * c, w.h, w.start1 + k0, bar);
    return;
  }
  const int psize = 1 << A.shift, rows = psize < KT ? psize : KT;
  const int32_t* table = A.table + (int64_t)w.b * A.width;
  for (int r = 0; r < KT; r += rows) {
    // pages behind the end, and page numbers outside the pool, arrive as zeros
    int page = (int)A.n_pages;
    if (k0 + r < w.len1) {
      const int32_t at = __ldg(table + ((k0 + r) >> A.shift));
      if (at >= 0 && at < A.n_pages) page = at;
      else atomicExch(&g_flash_fault, 1);
    }
    const int y = (w.h << A.shift) + ((k0 + r) & (psize - 1));
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      tma_load_3d(dst + c * BLK + r * 128, m, 64 * c, y, page, bar);
  }
}

// One warp: K and V of the tiles, in the order in which the products free their
// places (S 0, S 1, P V 0, S 2, P V 1, S 3, ...).  (In the order of the keys K of the
// tile after the next waited behind V of the next, and came late: 259 us against 248
// at 1560 rows x 40 heads over 8192 keys.)
//
// What it asks for first is on its way while the others still wait for TMEM.
template <int D>
__device__ __forceinline__ void load_role(const FlashArgs& A, uint8_t* smem, uint64_t* bars,
                                          const Work& w) {
  using L = Lay<D>;
  const int lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem);
  int rag = 0, done[2] = {0, 0};  // ragged tiles so far; tiles of K and V on their way
  if (A.qtma) {
    // boxes of 64 channels, the key head's g query heads and 128 / g tokens; rows of
    // no row of this CTA are computed with and not stored
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars[L::B_Q], L::Q_TILE);
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        tma_load_3d(base + c * (QT * 128), &A.q, 64 * c, w.h * A.g, (int)w.tok0 + w.token(A, w.r0),
                    &bars[L::B_Q]);
    }
    __syncwarp();
  }
  // K (v = 0) or V (v = 1) of tile t < w.n; whether its place came free
  auto load = [&](int t, int v) -> bool {
    const int at = t & 1;
    if (t >= 2 && !warp_wait(&bars[(v ? L::B_PV : L::B_S) + at], ((t >> 1) - 1) & 1)) return false;
    const int j = w.j0 + t;
    const int left = j < w.nt0 ? KT : w.len1 - (j - w.nt0) * KT;
    const uint32_t off = (v ? L::OFF_V : L::OFF_K) + at * L::ENT, dst = base + off;
    uint64_t* const full = &bars[(v ? L::B_V : L::B_K) + at];
    // V rows behind the end are overwritten before the tile is handed on
    const bool wipe = v && left < KT;
    uint64_t* bar = wipe ? &bars[L::B_RAG] : full;
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, L::ENT);
      issue_tile<D>(A, w, j, v, dst, bar);
    }
    __syncwarp();
    if (wipe) {
      if (!warp_wait(bar, rag++ & 1)) return false;
      constexpr int C = D / 8;
      for (int x = left * C + lane; x < KT * C; x += 32)
        *reinterpret_cast<uint4*>(smem + off + sw128_off(x / C, x % C, KT)) =
            make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      warp_arrive(full);
    }
    ++done[v];
    return true;
  };
  const int n = w.n;
  bool ok = true;
  for (int t = 0; t < 2 && t < n; ++t) load(t, 0);
  start_barrier();
  for (int t = 0; ok && t < 2 && t < n; ++t) ok = load(t, 1);
  if (ok && n > 2) ok = load(2, 0);
  for (int t = 2; ok && t < n; ++t) ok = (t + 1 >= n || load(t + 1, 0)) && load(t, 1);
  // every box issued has landed before the CTA may exit
  if (A.qtma && !warp_wait(&bars[L::B_Q], 0)) ok = false;
#pragma unroll
  for (int v = 0; v < 2; ++v)
    for (int t = done[v] > 2 ? done[v] - 2 : 0; t < done[v]; ++t)
      if (!warp_wait(&bars[(v ? L::B_V : L::B_K) + (t & 1)], (t >> 1) & 1)) ok = false;
  if (!ok && lane == 0) timeout_flag();
}

// ------------------------------------------------------------------ MMA role
// One warp: two tiles' S = Q K^T ahead, then for each tile O += P V and S of the
// tile after the next, into the buffer that P occupied (the tensor core works in
// issue order).  A commit tells when all before it is complete.
//
// The whole warp runs the role, on values that the compiler knows to be uniform and
// with the places of two tiles as constants, and one lane issues: a lane by itself
// spent 1250 cycles on the twelve products and two commits of a tile, moving
// descriptors, and bounded everything (1350 cycles per tile; the products take 643:
// 64 each for P V, and 48 each for S, whose 64 columns read 6 KB of shared memory).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

template <int D>
struct MmaWarp {
  using L = Lay<D>;
  uint64_t* bars;
  uint32_t tmem;
  uint64_t qd, kd, vd;
  bool leader;

  template <int AT>
  __device__ __forceinline__ void scores() const {  // S of the tile whose K lies in place AT
    constexpr uint32_t IDQ = idesc_bf16(QT, KT, false, false);
    tc_fence_after();
    if (leader) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t in = (k & 3) * 32;
        mma_bf16_ss(tmem + 64 * AT, qd + (((k >> 2) * (QT * 128) + in) >> 4),
                    kd + ((AT * L::ENT + (k >> 2) * (KT * 128) + in) >> 4), IDQ, k > 0);
      }
      mma_commit(&bars[L::B_S + AT]);
    }
    __syncwarp();
  }

  // O += P V of tile t in place AT, and S of tile t + 2
  template <int AT>
  __device__ __forceinline__ bool step(int t, int n) const {
    constexpr uint32_t IDP = idesc_bf16(QT, D, false, true);
    const uint32_t phase = (t >> 1) & 1;
    if (!warp_wait(&bars[L::B_V + AT], phase) || !warp_wait(&bars[L::B_P + AT], phase)) return false;
    tc_fence_after();
    if (leader) {
#pragma unroll
      for (int k = 0; k < KT / 16; ++k)
        mma_bf16_ts(tmem + 128, tmem + 64 * AT + 8 * k, vd + ((AT * L::ENT + k * 16 * 128) >> 4), IDP,
                    (k > 0 || t > 0) ? 1u : 0u);
      mma_commit(&bars[L::B_PV + AT]);
    }
    __syncwarp();
    if (t + 2 < n) {
      if (!warp_wait(&bars[L::B_K + AT], phase ^ 1)) return false;
      scores<AT>();
    }
    return true;
  }
};

template <int D>
__device__ __forceinline__ void mma_role(uint8_t* smem, uint64_t* bars, uint32_t tmem,
                                         const Work& w) {
  using L = Lay<D>;
  const uint32_t base = smem_u32(smem);
  MmaWarp<D> m;
  m.bars = bars;
  m.tmem = __shfl_sync(0xffffffffu, tmem, 0);
  m.qd = desc_sw128(base, 16, 1024);
  m.kd = desc_sw128(base + L::OFF_K, 16, 1024);
  // V: channels are the contiguous dimension; its 64-channel blocks lie KT * 128 bytes apart
  m.vd = desc_sw128(base + L::OFF_V, KT * 128, 1024);
  m.leader = elect_one();
  const int n = __shfl_sync(0xffffffffu, w.n, 0);
  bool ok = warp_wait(&bars[L::B_Q], 0) && warp_wait(&bars[L::B_K], 0);
  if (ok) m.template scores<0>();
  if (ok && n > 1) {
    ok = warp_wait(&bars[L::B_K + 1], 0);
    if (ok) m.template scores<1>();
  }
  for (int t = 0; ok && t < n; t += 2) {
    ok = m.template step<0>(t, n);
    if (ok && t + 1 < n) ok = m.template step<1>(t + 1, n);
  }
  if (m.leader) mma_commit(&bars[L::B_DONE]);
  __syncwarp();
  if (!warp_wait(&bars[L::B_DONE], 0)) ok = false;
  if (!ok && m.leader) timeout_flag();
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 2) flash_kernel(const __grid_constant__ FlashArgs A) {
  using L = Lay<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Work w;
  if (!work_of(A, w)) return;
  if (w.n == 0) {  // no keys in this range
    const int rr = threadIdx.x;
    for (int e = rr; e < w.nr * (D / 8); e += NTHREADS) {
      const int64_t row = out_row(A, w, w.r0 + e / (D / 8));
      const int c = e % (D / 8);
      if (A.part0 >= 0) {
        const size_t at = (size_t)w.part * A.nq * A.Hq + row;
        float4* dst = reinterpret_cast<float4*>(A.ws_o + at * D) + 2 * c;
        dst[0] = dst[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c == 0) A.ws_l[at] = -INFINITY;
      } else {
        reinterpret_cast<uint4*>(A.O + row * D)[c] = make_uint4(0, 0, 0, 0);
        if (c == 0 && A.lse) A.lse[row] = -INFINITY;
      }
    }
    return;
  }
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + L::OFF_BAR + L::NBAR * 8);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0);
  if (warp == W_LOAD) {
    const int b = threadIdx.x & 31;  // one each
    if (b < L::NBAR)
      mbar_init(&bars[b], b == L::B_P || b == L::B_P + 1 ? (w.nr + 31) / 32 : b == L::B_Q && !A.qtma ? W_LOAD : 1);
    fence_mbar_init();
    __syncwarp();
    load_role<D>(A, smem, bars, w);  // (passes the barrier below on its way)
  } else {
    if (warp == W_MMA) {
      tmem_alloc(holder, COLS);
      tmem_relinquish();
    }
    tc_fence_before();
    start_barrier();
    tc_fence_after();
    if (warp < W_LOAD) softmax_role<D>(A, smem, bars, *holder, w);
    else mma_role<D>(smem, bars, *holder, w);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(*holder, COLS);
  }
}

// Merge of `np` partials per (query row, head): one warp per row.  With L_c
// their log-sum-exps, O = sum_c e^(L_c - L) O_c / sum_c e^(L_c - L), L = max L_c;
// rows of no sequence, or beyond max_q, stay as they were.
template <int D>
__global__ void __launch_bounds__(256) merge_kernel(const float* __restrict__ ws_o,
                                                    const float* __restrict__ ws_l, int np,
                                                    int64_t nq, int Hq,
                                                    const int32_t* __restrict__ cu, int64_t n_seq,
                                                    int64_t max_q, uint16_t* __restrict__ O,
                                                    float* __restrict__ lse) {
  const int64_t rows = nq * Hq;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int lane = threadIdx.x & 31;
  const int64_t t = row / Hq;
  // the last sequence that begins at or before t, 32 probes at a time
  int64_t lo = -1, hi = n_seq + 1;
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 31) / 32, x = lo + (lane + 1) * step;
    const unsigned below = __ballot_sync(0xffffffffu, x < hi && __ldg(cu + x) <= t);
    const int n = below == 0xffffffffu ? 32 : __ffs(~below) - 1;  // the leading probes
    const int64_t up = lo + (n + 1) * step;
    lo += n * step;
    hi = up < hi ? up : hi;
  }
  if (lo < 0 || lo >= n_seq) return;
  const int64_t c0 = __ldg(cu + lo), c1 = __ldg(cu + lo + 1);
  if (t - c0 >= max_q || c0 < 0 || c1 > nq || c1 <= t) return;
  // (at most 64 partials: two of their weights per lane)
  float l0 = lane < np ? __ldg(ws_l + (size_t)lane * rows + row) : -INFINITY;
  float l1 = lane + 32 < np ? __ldg(ws_l + (size_t)(lane + 32) * rows + row) : -INFINITY;
  float L = fmaxf(l0, l1);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L = fmaxf(L, __shfl_xor_sync(0xffffffffu, L, o));
  if (__any_sync(0xffffffffu, l0 != l0 || l1 != l1)) L = NAN;  // (the maximum leaves a NaN out)
  constexpr int V = D / 32;
  float acc[V], den = 0.0f;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.0f;
  if (L != -INFINITY) {
    const float w0 = expf(l0 - L), w1 = expf(l1 - L);
#pragma unroll 4
    for (int c = 0; c < np; ++c) {
      const float wt = __shfl_sync(0xffffffffu, c < 32 ? w0 : w1, c & 31);
      const float* o = ws_o + ((size_t)c * rows + row) * D + V * lane;
      den += wt;
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        float2 x = make_float2(0.0f, 0.0f);
        if (wt != 0.0f) x = __ldg(reinterpret_cast<const float2*>(o + e));  // (an empty partial's values are not written)
        acc[e] = fmaf(wt, x.x, acc[e]);
        acc[e + 1] = fmaf(wt, x.y, acc[e + 1]);
      }
    }
  }
  const float inv = den == 0.0f ? 0.0f : 1.0f / den;
#pragma unroll
  for (int e = 0; e < V; e += 2)
    *reinterpret_cast<uint32_t*>(O + row * D + V * lane + e) =
        pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (lse && lane == 0) lse[row] = den == 0.0f ? -INFINITY : L + logf(den);
}

// ------------------------------------------------------------------ host side
int device_sms() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 148;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// How a launch divides its work: row blocks per sequence, key ranges per row block.
struct Blocks {
  int qblocks, nsplit;
  double cost;  // in key tiles of a CTA
};

// rows: of a sequence; units: sequences times key heads; ntile: key tiles; most:
// key ranges at most; merged: the result is a partial in any case.  The key ranges
// are the count that minimizes (rounds of CTAs on the GPU) x (tiles per range + a
// fixed cost of 8 tiles) + 8 tiles for a merge's launch that one range does not need:
// a tile of few rows takes 0.76 us (eight single rows x 12 heads over 512 keys: 12.3
// us whole, 15.2 us in two ranges; over 1000 keys 18.4 us whole, 17.8 us in three).
Blocks blocks_of(int64_t rows, int64_t units, int64_t ntile, int most, bool merged) {
  Blocks b;
  b.qblocks = (int)((rows + QT - 1) / QT);
  const int64_t ctas = units * b.qblocks, slots = 2 * (int64_t)device_sms();
  b.nsplit = 1;
  b.cost = 1e300;
  for (int s = 1; s <= most && s * 4 <= (ntile > 4 ? ntile : 4); ++s) {
    const double c = (double)((ctas * s + slots - 1) / slots) * ((double)ntile / s + 8.0) +
                     (merged || s > 1 ? 8.0 : 0.0);
    if (c < b.cost * 0.98) {
      b.cost = c;
      b.nsplit = s;
    }
  }
  return b;
}

// The driver's encoder of tensor maps (no link to the driver library).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (EncodeFn)f;
  }();
  return fn;
}

// Map of bf16 [n2][n1][D] with the given distances in elements; boxes of 64
// channels by b1 by b2, 128-byte swizzle.
bool map_3d(CUtensorMap* m, const void* base, int D, int64_t n1, int64_t ld1, int64_t n2, int64_t ld2,
            int b1, int b2) {
  const EncodeFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)n1, (cuuint64_t)n2};
  const cuuint64_t strides[2] = {(cuuint64_t)ld1 * 2, (cuuint64_t)ld2 * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)b1, (cuuint32_t)b2};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Q's map, where whole tokens make up a Q tile.
bool map_q(FlashArgs& a, int D) {
  a.qtma = QT % a.g == 0;
  return !a.qtma || map_3d(&a.q, a.Q, D, a.Hq, D, a.nq, a.ldq, a.g, QT / a.g);
}

template <int D>
cudaError_t launch_flash(const FlashArgs& a, int heads, int64_t n_seq, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(flash_kernel<D>, allowed, (int)Lay<D>::SMEM);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((int64_t)a.qblocks * a.nsplit), (unsigned)heads, (unsigned)n_seq);
  flash_kernel<D><<<grid, NTHREADS, Lay<D>::SMEM, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_flash(int D, const FlashArgs& a, int heads, int64_t n_seq, cudaStream_t s) {
  return D == 128 ? launch_flash<128>(a, heads, n_seq, s) : launch_flash<64>(a, heads, n_seq, s);
}

cudaError_t launch_merge(int D, const FlashArgs& a, int np, const int32_t* cu, int64_t n_seq,
                         int64_t max_q, cudaStream_t s) {
  const unsigned grid = (unsigned)((a.nq * a.Hq + 7) / 8);
  if (D == 128)
    merge_kernel<128><<<grid, 256, 0, s>>>(a.ws_o, a.ws_l, np, a.nq, a.Hq, cu, n_seq, max_q, a.O, a.lse);
  else
    merge_kernel<64><<<grid, 256, 0, s>>>(a.ws_o, a.ws_l, np, a.nq, a.Hq, cu, n_seq, max_q, a.O, a.lse);
  return cudaGetLastError();
}

constexpr int64_t kMaxGridX = (int64_t(1) << 31) - 1;

// Partials that a call may use: as many as 64 MiB hold, 64 at most.
int partials_of(int64_t n_q, int Hq, int d) {
  const int64_t one = n_q * Hq * (d + 1) * 4;
  if (one <= 0) return 0;
  const int64_t n = (int64_t(64) << 20) / one;
  return (int)(n > 64 ? 64 : n);
}

size_t partial_bytes(int np, int64_t n_q, int Hq, int d) {
  return ((size_t)np * n_q * Hq * (d + 1) * 4 + 255) / 256 * 256;
}

// How a shared-history call runs.  joined: one CTA takes its rows through the
// history and then through its branch's own keys.  Otherwise all branches' rows
// pack into common row blocks for the history, which few rows per branch would
// leave mostly empty, the own keys follow per branch, and the two are merged (two
// partials, however large).
// With few rows in all the history is not unpacked at all (attention_rows.cu).
// Between the first two the costs of blocks_of decide.
struct SharedPlan {
  bool rows, joined;
  int np;          // partials that the workspace holds
  Blocks all;      // joined
  Blocks own;      // not joined; no key range: no own keys
  Blocks history;  // not joined, not rows
};

SharedPlan plan_shared(const Dims& D, int64_t T, int Hq, int64_t n_q, int64_t n_seq, int64_t max_q,
                       int64_t max_kv) {
  SharedPlan p = {};
  const int g = Hq / D.H;
  const int64_t mq = max_q < n_q ? max_q : n_q;
  const int64_t tiles0 = (T + KT - 1) / KT, tiles1 = (max_kv + KT - 1) / KT;
  p.np = partials_of(n_q, Hq, D.d);
  p.rows = p.np >= 8 && rows_supported(D, T, n_q * g, device_sms());
  p.all = blocks_of(mq * g, D.H * n_seq, tiles0 + tiles1, p.np < 2 ? 1 : p.np, false);
  if (p.rows || T > 0) {
    const int np = p.np < 2 ? 2 : p.np;
    double cost = 0.0;
    if (max_kv > 0) {
      p.own = blocks_of(mq * g, D.H * n_seq, tiles1, np / 2, true);
      cost = p.own.cost;
    }
    p.history = blocks_of(n_q * g, D.H, tiles0, np - p.own.nsplit, true);
    p.joined = !p.rows && p.all.cost <= cost + p.history.cost;
    if (!p.joined) p.np = np;
  } else {
    p.joined = true;
  }
  return p;
}

bool lengths_ok(int64_t n_q, int g, int Hq, int64_t n_seq, int64_t max_q, int64_t max_kv) {
  return n_q >= 0 && n_q * g <= kMostKeys && n_q * Hq <= 8 * kMaxGridX && n_seq >= 1 && n_seq <= 65535 &&
         max_q >= 0 && max_q <= kMaxGridX && max_kv >= 0 && max_kv <= kMostKeys;
}

}  // namespace

int read_and_clear_flash_timeout() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_flash_timeout, sizeof(int)) != cudaSuccess) return -1;
  if (v) cudaMemcpyToSymbol(g_flash_timeout, &z, sizeof(int));
  return v;
}

int read_and_clear_flash_fault() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_flash_fault, sizeof(int)) != cudaSuccess) return -1;
  if (v) cudaMemcpyToSymbol(g_flash_fault, &z, sizeof(int));
  return v;
}

}  // namespace qwm

using namespace qwm;

extern "C" qwm_status qwm_attention_shared_workspace(const qwm_cache* c, int64_t n_q,
                                                     int32_t heads_q, int64_t n_seq, int64_t max_q,
                                                     int64_t max_kv, uint64_t* least,
                                                     uint64_t* full) {
  if (!cache_ok(c) || c->len > kMostKeys || !least || !full || heads_q < 1 || heads_q > 65535 || heads_q % c->cfg.heads ||
      !lengths_ok(n_q, heads_q / c->cfg.heads, heads_q, n_seq, max_q, max_kv))
    return QWM_ERR_INVALID_ARG;
  *least = *full = 0;
  if (n_q == 0 || max_q == 0) return QWM_OK;
  const Dims D = dims_of(&c->cfg);
  const SharedPlan p = plan_shared(D, c->len, heads_q, n_q, n_seq, max_q, max_kv);
  const uint64_t head = p.rows ? 0 : (uint64_t)c->len * D.d * 4;
  const uint64_t part = partial_bytes(p.np, n_q, heads_q, D.d);
  *least = part + head;
  *full = part + head * D.H;
  return QWM_OK;
}

extern "C" qwm_status qwm_attention_shared(const qwm_cache* c, const void* Q, int64_t ldq,
                                           int64_t n_q, int32_t heads_q, const int32_t* cu,
                                           int64_t n_seq, int64_t max_q, const qwm_pages* pages,
                                           const int32_t* table, int32_t table_width,
                                           const int32_t* kv_len, int64_t max_kv, int32_t causal,
                                           float scale, void* O, float* lse, void* workspace,
                                           uint64_t workspace_bytes, void* stream) {
  uint64_t least = 0, full = 0;
  const qwm_status st =
      qwm_attention_shared_workspace(c, n_q, heads_q, n_seq, max_q, max_kv, &least, &full);
  if (st != QWM_OK) return st;
  const Dims D = dims_of(&c->cfg);
  if (!cu || (n_q > 0 && (!Q || !O)) || ldq < (int64_t)heads_q * D.d || ldq % 8)
    return QWM_ERR_INVALID_ARG;
  if (pages) {
    if (!pages_ok(pages) || pages->heads != D.H || pages->head_dim != D.d || !table || !kv_len ||
        table_width < 1)
      return QWM_ERR_INVALID_ARG;
  } else if (max_kv > 0) {
    return QWM_ERR_INVALID_ARG;
  }
  if (!aligned_to(Q, 16) || !aligned_to(O, 16) || !aligned_to(lse, 4) || !aligned_to(cu, 4) ||
      !aligned_to(table, 4) || !aligned_to(kv_len, 4) || !aligned_to(workspace, 256) ||
      (pages && (!aligned_to(pages->K, 16) || !aligned_to(pages->V, 16))))
    return QWM_ERR_ALIGNMENT;
  if (c->len > 0 && !c->has_centroids) return QWM_ERR_STATE;
  if (n_q == 0 || max_q == 0) return QWM_OK;
  if (workspace_bytes < least || (least > 0 && !workspace)) return QWM_ERR_CAPACITY;

  const int g = heads_q / D.H;
  const int64_t T = c->len;
  SharedPlan plan = plan_shared(D, T, heads_q, n_q, n_seq, max_q, max_kv);
  const CacheView v = view_of(c);
  const cudaStream_t s = (cudaStream_t)stream;
  FlashArgs a = {};
  a.Q = (const uint16_t*)Q;
  a.ldq = ldq;
  a.nq = n_q;
  a.Hq = heads_q;
  a.g = g;
  a.max_q = max_q;
  a.scale_log2 = (scale > 0.0f ? scale : 1.0f / sqrtf((float)D.d)) * 1.4426950408889634f;
  a.O = (uint16_t*)O;
  a.lse = lse;
  a.ws_o = (float*)workspace;
  a.ws_l = a.ws_o + (size_t)plan.np * n_q * heads_q * D.d;
  if (!map_q(a, D.d)) return QWM_ERR_CUDA;
  uint8_t* scratch = (uint8_t*)workspace + partial_bytes(plan.np, n_q, heads_q, D.d);
  // the branches' own keys
  FlashArgs own = a;
  own.cu = cu;
  own.causal = causal != 0;
  if (pages) {
    own.own = OWN_PAGES;
    const int64_t rows = (int64_t)pages->heads * pages->page_size;
    const int box = pages->page_size < KT ? pages->page_size : KT;
    if (max_kv > 0 &&
        (!map_3d(&own.k1, pages->K, D.d, rows, D.d, pages->n_pages, rows * D.d, box, 1) ||
         !map_3d(&own.v1, pages->V, D.d, rows, D.d, pages->n_pages, rows * D.d, box, 1)))
      return QWM_ERR_CUDA;
    own.kv_len = kv_len;
    own.table = table;
    own.max_kv = max_kv;
    own.n_pages = pages->n_pages;
    own.width = table_width;
    own.shift = page_shift(pages);
  }
  // heads per pass: what the workspace holds unpacked
  const uint64_t head = plan.rows ? 0 : (uint64_t)T * D.d * 4;
  int hp = D.H;
  if (head > 0) {
    const uint64_t fit = (workspace_bytes - (uint64_t)(scratch - (uint8_t*)workspace)) / head;
    hp = fit < (uint64_t)D.H ? (int)fit : D.H;
  }
  // passes of even size
  const int passes = (D.H + hp - 1) / hp;
  hp = (D.H + passes - 1) / passes;
  const int64_t mq = max_q < n_q ? max_q : n_q;
  const int64_t tiles0 = (T + KT - 1) / KT, tiles1 = (max_kv + KT - 1) / KT;
  if (passes > 1) {
    plan.all = blocks_of(mq * g, hp * n_seq, tiles0 + tiles1, plan.np < 2 ? 1 : plan.np, false);
    plan.history = blocks_of(n_q * g, hp, tiles0, plan.np - plan.own.nsplit, true);
  }
  int np = 0;
  const auto set = [](FlashArgs& f, const Blocks& b) {
    f.qblocks = b.qblocks;
    f.nsplit = b.nsplit;
  };
  if (plan.joined) {
    set(own, plan.all);
    np = own.nsplit > 1 ? own.nsplit : 0;
    own.part0 = np > 0 ? 0 : -1;
  } else {
    set(own, plan.own);
    if (plan.rows) {
      const RowsPlan rp = rows_plan(D, T, device_sms(), plan.np - own.nsplit);
      a.nsplit = rp.slots;
      if (launch_rows(D, v, T, a.Q, ldq, n_q, heads_q, a.scale_log2, rp, a.ws_o, a.ws_l, s) != cudaSuccess)
        return QWM_ERR_CUDA;
    } else {
      a.max_q = n_q;
      set(a, plan.history);
    }
    a.part0 = 0;
    own.part0 = a.nsplit;
    np = a.nsplit + own.nsplit;
  }
  FlashArgs& with0 = plan.joined ? own : a;
  for (int h0 = 0; h0 < D.H && !plan.rows; h0 += hp) {
    const int nh = D.H - h0 < hp ? D.H - h0 : hp;
    if (T > 0) {
      uint16_t* const K0 = (uint16_t*)scratch;
      uint16_t* const V0 = K0 + (size_t)nh * T * D.d;
      with0.len0 = T;
      if (!map_3d(&with0.k0, K0, D.d, T, D.d, nh, T * D.d, KT, 1) ||
          !map_3d(&with0.v0, V0, D.d, T, D.d, nh, T * D.d, KT, 1) ||
          launch_unpack(D, v, T, h0, nh, K0, V0, device_sms(), s) != cudaSuccess)
        return QWM_ERR_CUDA;
    }
    with0.head0 = h0;
    if (launch_flash(D.d, with0, nh, plan.joined ? n_seq : 1, s) != cudaSuccess) return QWM_ERR_CUDA;
  }
  if (!plan.joined && own.nsplit > 0 && launch_flash(D.d, own, D.H, n_seq, s) != cudaSuccess)
    return QWM_ERR_CUDA;
  if (np > 0 && launch_merge(D.d, a, np, cu, n_seq, max_q, s) != cudaSuccess) return QWM_ERR_CUDA;
  return QWM_OK;
}

extern "C" qwm_status qwm_cross_attention_workspace(int32_t heads_q, int32_t heads_kv,
                                                    int32_t head_dim, int64_t n_q, int64_t n_seq,
                                                    int64_t max_q, int64_t max_kv, uint64_t* least,
                                                    uint64_t* full) {
  if (!least || !full || heads_kv < 1 || heads_q < 1 || heads_q > 65535 || heads_q % heads_kv ||
      (head_dim != 64 && head_dim != 128) ||
      !lengths_ok(n_q, heads_q / heads_kv, heads_q, n_seq, max_q, max_kv))
    return QWM_ERR_INVALID_ARG;
  const int64_t mq = max_q < n_q ? max_q : n_q;
  const int np = blocks_of(mq * (heads_q / heads_kv), heads_kv * n_seq, (max_kv + KT - 1) / KT,
                           partials_of(n_q, heads_q, head_dim), false)
                     .nsplit;
  *least = 0;
  *full = np > 1 ? partial_bytes(np, n_q, heads_q, head_dim) : 0;
  return QWM_OK;
}

extern "C" qwm_status qwm_cross_attention(const void* Q, int64_t ldq, int64_t n_q, int32_t heads_q,
                                          const void* K, int64_t ldk, const void* V, int64_t ldv,
                                          int64_t n_kv, int32_t heads_kv, int32_t head_dim,
                                          const int32_t* cu, const int32_t* kv_start,
                                          const int32_t* kv_len, int64_t n_seq, int64_t max_q,
                                          int64_t max_kv, float scale, void* O, float* lse,
                                          void* workspace, uint64_t workspace_bytes, void* stream) {
  uint64_t least = 0, full = 0;
  const qwm_status st = qwm_cross_attention_workspace(heads_q, heads_kv, head_dim, n_q, n_seq, max_q,
                                                      max_kv, &least, &full);
  if (st != QWM_OK) return st;
  if (!cu || !kv_start || !kv_len || (n_q > 0 && (!Q || !O)) || n_kv < 0 || n_kv > kMostKeys ||
      (n_kv > 0 && max_kv > 0 && (!K || !V)) || ldq < (int64_t)heads_q * head_dim || ldq % 8 ||
      ldk < (int64_t)heads_kv * head_dim || ldk % 8 || ldv < (int64_t)heads_kv * head_dim || ldv % 8)
    return QWM_ERR_INVALID_ARG;
  if (!aligned_to(Q, 16) || !aligned_to(K, 16) || !aligned_to(V, 16) || !aligned_to(O, 16) ||
      !aligned_to(lse, 4) || !aligned_to(cu, 4) || !aligned_to(kv_start, 4) ||
      !aligned_to(kv_len, 4) || !aligned_to(workspace, 256))
    return QWM_ERR_ALIGNMENT;
  if (n_q == 0 || max_q == 0) return QWM_OK;
  const int g = heads_q / heads_kv;
  const int64_t mq = max_q < n_q ? max_q : n_q;
  FlashArgs a = {};
  a.Q = (const uint16_t*)Q;
  a.ldq = ldq;
  a.nq = n_q;
  a.Hq = heads_q;
  a.g = g;
  if (!map_q(a, head_dim)) return QWM_ERR_CUDA;
  a.cu = cu;
  a.max_q = max_q;
  a.own = OWN_ROWS;
  a.n_kv = n_kv;
  if (n_kv > 0 && max_kv > 0 &&
      (!map_3d(&a.k1, K, head_dim, heads_kv, head_dim, n_kv, ldk, 1, KT) ||
       !map_3d(&a.v1, V, head_dim, heads_kv, head_dim, n_kv, ldv, 1, KT)))
    return QWM_ERR_CUDA;
  a.kv_start = kv_start;
  a.kv_len = kv_len;
  a.max_kv = max_kv;
  a.scale_log2 = (scale > 0.0f ? scale : 1.0f / sqrtf((float)head_dim)) * 1.4426950408889634f;
  a.O = (uint16_t*)O;
  a.lse = lse;
  const bool parts = full > 0 && workspace && workspace_bytes >= full;
  const Blocks b = blocks_of(mq * g, heads_kv * n_seq, (max_kv + KT - 1) / KT,
                             parts ? partials_of(n_q, heads_q, head_dim) : 1, false);
  a.qblocks = b.qblocks;
  a.nsplit = b.nsplit;
  a.part0 = -1;
  if (parts) {
    a.part0 = 0;
    a.ws_o = (float*)workspace;
    a.ws_l = a.ws_o + (size_t)b.nsplit * n_q * heads_q * head_dim;
  }
  const cudaStream_t s = (cudaStream_t)stream;
  if (launch_flash(head_dim, a, heads_kv, n_seq, s) != cudaSuccess) return QWM_ERR_CUDA;
  if (a.nsplit > 1 && launch_merge(head_dim, a, a.nsplit, cu, n_seq, max_q, s) != cudaSuccess)
    return QWM_ERR_CUDA;
  return QWM_OK;
}
