// Orthogonalised updates by Newton-Schulz products: the optimiser step on
// packed skew blocks (poetx_muon_step_batch) and dense matrices
// (poetx_orthogonalize).
//
//   X_0 = M / (|M|_F + eps);  A = X X^T;  B = b A + c A^2;  X <- a X + B X
//
// maps every singular value s of X to p(s) = a s + b s^3 + c s^5 and keeps the
// singular vectors, so a few steps with a suitable p bring all of them near 1.
//
// Operands.  X, A and B live in the workspace as fp16 "planes" at a fixed power
// of two: hi = fp16(x), lo = fp16(x - hi), 22 bits together.  The products run
// on the fp16 matrix instructions with fp32 accumulation.  With NP = 3 a
// product is hi hi + hi lo + lo hi: as exact as fp32 products (the low-by-low
// part is 2^-22 of the whole) at three times the cost of one, about 5x the rate
// of the fp32 matrix instructions; packed parameters and fp32 matrices take it.
// With NP = 1 (bf16 matrices) it is hi hi, and only the term a X is carried in
// both planes: measured against the definition in 64 bits the result is off by
// 1.2 to 2.4e-3 of its norm before the rounding to bf16, which is off by 1.7e-3
// itself (bf16 products would be off by 1 to 2e-2).
//
// Scales: X is held times SX, a power of two near 8 sqrt(K) for rows of length
// K (an orthogonal result has entries near K^-1/2), A and B times SA = 2^8.
// The host refuses coefficients whose p takes a singular value out of the range
// that keeps every entry within fp16.
//
// Symmetry.  A and B are symmetric; for skew M every X is skew, so X^T = -X
// and all three products read rows only: A = X X^T, A^2 = A A^T,
// B X = -(B X^T).  Their tiles on and above the diagonal are computed and
// written twice, the second time transposed (negated for X): (n + 1) / 2n of
// the tiles.  Dense X is kept in both orientations instead.
//
// Every buffer is padded with zeros to whole tiles, so the K loop copies 16
// bytes a lane straight into LDS with no bounds.
#include <cmath>
#include <cstddef>

#include "kernel_util.h"

using namespace px;

namespace {

typedef _Float16 f16;
typedef _Float16 f16x8_v __attribute__((ext_vector_type(8)));

constexpr float kSA = 256.f;  // scale of A and B

// Tile configuration of the product kernels.  PL planes per operand.
template <int BM_, int BN_, int BK_, int WM_, int WN_, int NP_> struct NCfg {
  static constexpr int BM = BM_, BN = BN_, BK = BK_, WM = WM_, WN = WN_, NP = NP_, PL = NP_ == 3 ? 2 : 1;
  static constexpr int NW = WM * WN, NT = NW * 64;
  static constexpr int WTM = BM / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
  static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2;  // one plane of one stage
  static constexpr int STAGE = PL * (A_BYTES + B_BYTES);
  // the epilogue stages RS rows of (hi, lo) words; a pitch of 5 mod 64 words spreads both the reads
  // along its rows and those down its columns over the banks
  static constexpr int RS = 128, PITCH = BN + 5, EPI = RS * PITCH * 4;
  static constexpr int LDS = 2 * STAGE > EPI ? 2 * STAGE : EPI;
  static_assert(A_BYTES % (1024 * NW) == 0 && B_BYTES % (1024 * NW) == 0, "tile must split into 1 KB per wave");
  static_assert(BM % RS == 0 && RS % WTM == 0 && PITCH % 64 == 5, "epilogue stage");
};
template <int NP> using NSmall = NCfg<128, 128, NP == 3 ? 32 : 64, 2, 2, NP>;  // 4 waves of 64 x 64, two workgroups a CU
template <int NP> using NBig = NCfg<256, 256, NP == 3 ? 32 : 64, 4, 2, NP>;    // 8 waves of 64 x 128

PX_DEV f16x8_v as_f16(const bf16x8_v& x) {
  f16x8_v y;
  __builtin_memcpy(&y, &x, 16);
  return y;
}

PX_DEV uint32_t pack_hilo(float v) {
  const f16 h = (f16)v, l = (f16)(v - (float)h);
  uint16_t hb, lb;
  __builtin_memcpy(&hb, &h, 2);
  __builtin_memcpy(&lb, &l, 2);
  return (uint32_t)hb | ((uint32_t)lb << 16);
}

// One operand: K-contiguous rows of hi (and lo) values, ld elements apart.
struct Planes {
  f16 *h = nullptr, *l = nullptr;
  int64_t ld = 0, stride = 0;  // stride: elements from one matrix of the batch to the next
  PX_DEV Planes at(int z, int64_t row) const {
    const int64_t o = z * stride + row * ld;
    return Planes{h + o, l ? l + o : nullptr, ld, stride};
  }
  PX_DEV Planes tile(int z, int row, int col) const { return h ? at(z, row).right(col) : *this; }
  PX_DEV Planes right(int col) const { return Planes{h + col, l ? l + col : nullptr, ld, stride}; }
};

// acc = sum over KT tiles of K of a's tile rows times b's tile rows.  `same`: the two tiles are one.
template <class C> PX_DEV void ns_loop(char* lds, const Planes& a, const Planes& b, int KT, bool same, Acc<C>& acc) {
  const AccPos<C> p = acc_pos<C>();
  const int wave = threadIdx.x >> 6, lane = p.lane;
  auto issue = [&](int kt, char* st) {
    const int k0 = kt * C::BK;
    dma_kmaj<C::BM, C::BK, C::NW>(reinterpret_cast<const bf16_t*>(a.h), a.ld, k0, st, wave, lane);
    if constexpr (C::PL == 2)
      dma_kmaj<C::BM, C::BK, C::NW>(reinterpret_cast<const bf16_t*>(a.l), a.ld, k0, st + C::A_BYTES, wave, lane);
    if (same) return;
    st += C::PL * C::A_BYTES;
    dma_kmaj<C::BN, C::BK, C::NW>(reinterpret_cast<const bf16_t*>(b.h), b.ld, k0, st, wave, lane);
    if constexpr (C::PL == 2)
      dma_kmaj<C::BN, C::BK, C::NW>(reinterpret_cast<const bf16_t*>(b.l), b.ld, k0, st + C::B_BYTES, wave, lane);
  };
  acc.zero();
  if (KT > 0) issue(0, lds);
  for (int kt = 0; kt < KT; ++kt) {
    wait_vm<0>();
    wait_lgkm0();
    barrier_raw();
    if (kt + 1 < KT) issue(kt + 1, lds + ((kt + 1) & 1) * C::STAGE);
    const char* As = lds + (kt & 1) * C::STAGE;
    const char* Bs = same ? As : As + C::PL * C::A_BYTES;
    const int bpl = same ? C::A_BYTES : C::B_BYTES;
#pragma unroll
    for (int ks = 0; ks < C::BK / 16; ++ks) {
      f16x8_v ah[C::TM], bh[C::TN], al[C::PL == 2 ? C::TM : 1], bl[C::PL == 2 ? C::TN : 1];
#pragma unroll
      for (int i = 0; i < C::TM; ++i) {
        const int t0 = p.wm * C::WTM + i * 32;
        ah[i] = as_f16(frag_kmaj<C::BK>(As, t0, ks * 16, lane));
        if constexpr (C::PL == 2) al[i] = as_f16(frag_kmaj<C::BK>(As + C::A_BYTES, t0, ks * 16, lane));
      }
#pragma unroll
      for (int j = 0; j < C::TN; ++j) {
        const int t0 = p.wn * C::WTN + j * 32;
        bh[j] = as_f16(frag_kmaj<C::BK>(Bs, t0, ks * 16, lane));
        if constexpr (C::PL == 2) bl[j] = as_f16(frag_kmaj<C::BK>(Bs + bpl, t0, ks * 16, lane));
      }
#pragma unroll
      for (int i = 0; i < C::TM; ++i)
#pragma unroll
        for (int j = 0; j < C::TN; ++j) {
          if constexpr (C::PL == 2) {
            acc.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(al[i], bh[j], acc.v[i][j], 0, 0, 0);
            acc.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah[i], bl[j], acc.v[i][j], 0, 0, 0);
          }
          acc.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah[i], bh[j], acc.v[i][j], 0, 0, 0);
        }
    }
  }
  wait_lgkm0();
  barrier_raw();
}

PX_DEV float plane_value(f16 h, f16 l) { return (float)h + (float)l; }

// 8 (hi, lo) words -> their hi and their lo halves, each flipped by x
PX_DEV void split_words(const uint32_t (&w)[8], uint32_t x, uint4& h, uint4& l) {
  uint32_t hh[4], ll[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    hh[e] = ((w[2 * e] & 0xffff) | (w[2 * e + 1] << 16)) ^ x;
    ll[e] = ((w[2 * e] >> 16) | (w[2 * e + 1] & 0xffff0000u)) ^ x;
  }
  h = make_uint4(hh[0], hh[1], hh[2], hh[3]);
  l = make_uint4(ll[0], ll[1], ll[2], ll[3]);
}

// The epilogue of a tile, v = alpha aux + beta acc, RS rows at a time through LDS: the accumulators are staged in
// fp32, then each thread takes 8 consecutive values of a row, adds the aux planes' (16-byte loads; null: none),
// writes them to the planes `o` (null: none) and leaves them in LDS, as (hi, lo) words where `t` (the transposed
// tile's planes; null: none) is written from there with `flip` (0x8000 negates), as floats for emit(r0, stage).
// All planes are at the tile's origin; null lo planes are skipped.
template <class C, class Emit>
PX_DEV void ns_store(char* lds, const Acc<C>& acc, const Planes& aux, float alpha, float beta, const Planes& o,
                     const Planes& t, uint32_t flip, const Emit& emit) {
  constexpr bool EMIT = !std::is_same<Emit, std::nullptr_t>::value;
  uint32_t* st = reinterpret_cast<uint32_t*>(lds);
  const AccPos<C> p = acc_pos<C>();
#pragma unroll 1
  for (int r0 = 0; r0 < C::BM; r0 += C::RS) {
    __syncthreads();
    if (p.wm * C::WTM / C::RS * C::RS == r0) {
#pragma unroll
      for (int i = 0; i < C::TM; ++i)
#pragma unroll
        for (int j = 0; j < C::TN; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            st[(p.row(i, e) - r0) * C::PITCH + p.col(j)] = __float_as_uint(beta * acc.v[i][j][e]);
    }
    __syncthreads();
#pragma unroll 2
    for (int c = threadIdx.x; c < C::RS * C::BN / 8; c += C::NT) {
      const int i = c / (C::BN / 8), j = c % (C::BN / 8) * 8;
      uint32_t* w = st + i * C::PITCH + j;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
      if (aux.h) {
        const int64_t at = (r0 + i) * aux.ld + j;
        const f16x8_v xh = *reinterpret_cast<const f16x8_v*>(aux.h + at);
        f16x8_v xl = {};
        if (aux.l) xl = *reinterpret_cast<const f16x8_v*>(aux.l + at);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += alpha * plane_value(xh[e], xl[e]);
      }
      if constexpr (EMIT) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(v[e]);
      } else {
        uint32_t x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = pack_hilo(v[e]);
        uint4 h, l;
        split_words(x, 0, h, l);
        const int64_t at = (r0 + i) * o.ld + j;
        *reinterpret_cast<uint4*>(o.h + at) = h;
        if (o.l) *reinterpret_cast<uint4*>(o.l + at) = l;
        if (t.h)
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = x[e];
      }
    }
    if constexpr (EMIT) {
      __syncthreads();
      emit(r0, reinterpret_cast<const float*>(st));
    } else if (t.h) {
      __syncthreads();
#pragma unroll 2
      for (int c = threadIdx.x; c < C::RS * C::BN / 8; c += C::NT) {
        const int j = c / (C::RS / 8), i = c % (C::RS / 8) * 8;
        uint32_t x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = st[(i + e) * C::PITCH + j];
        uint4 h, l;
        split_words(x, flip | (flip << 16), h, l);
        const int64_t at = j * t.ld + r0 + i;
        *reinterpret_cast<uint4*>(t.h + at) = h;
        if (t.l) *reinterpret_cast<uint4*>(t.l + at) = l;
      }
    }
  }
}

// Consecutive workgroups go to the 8 XCDs in turn: each XCD takes a contiguous range of units.
PX_DEV int xcd_unit(int id, int units) {
  const int x = id % 8, k = id / 8, q = units / 8, r = units % 8;
  return x * q + min(x, r) + k;
}

// u-th tile on or above the diagonal of n x n tiles, by rows
PX_DEV void upper_tile(int u, int n, int& ti, int& tj) {
  ti = 0;
  while (u >= n - ti) u -= n - ti++;
  tj = ti + u;
}

// The sides of a step on packed skew parameters: side s owns blocks [first[s], first[s + 1]).
struct MuonTable {
  float* q[pxk::kMaxSides];
  const float* g[pxk::kMaxSides];
  float* m[pxk::kMaxSides];
  int d[pxk::kMaxSides];
  int first[pxk::kMaxSides + 1];
  int count;
  // block z: its side, the first packed slot of it in the side's arrays, its live size
  PX_DEV void at(int z, int b, int& s, int64_t& off, int& r) const {
    s = 0;
    while (s + 1 < count && z >= first[s + 1]) ++s;
    const int blk = z - first[s];
    off = blk * ((int64_t)b * (b - 1) / 2);
    r = min(b, d[s] - blk * b);
  }
};

struct MuonK {
  float lr, wd, beta, omb, rms, eps;
  int nesterov;
  PX_DEV float moment(float m, float g) const { return beta * m + omb * g; }
  PX_DEV float update(float m, float g) const { return nesterov ? beta * m + omb * g : m; }
  // q <- q - lr (scale O + wd q)
  PX_DEV float step(float q, float o, float scale) const { return q - lr * (scale * o + wd * q); }
  PX_DEV float scale(int r) const { return rms > 0.f ? rms * __builtin_sqrtf((float)r) : 1.f; }
};

// ------------------------------------------------------------ skew blocks ---

// Momentum of every live slot, and each workgroup's sum of the squared updates
// in 64 bits: workgroup c of block z takes the packed rows c, c + gridDim.x, ...
// of waves.  A dead slot (j >= r of a partial block) is neither read nor written.
__global__ __launch_bounds__(256) void k_muon_momentum(MuonTable tab, int b, MuonK k, double* __restrict__ part) {
  __shared__ double red[4];
  const int z = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s, r;
  int64_t off;
  tab.at(z, b, s, off, r);
  const float* g = tab.g[s] + off;
  float* m = tab.m[s] + off;
  double sum = 0.0;
  for (int i = blockIdx.x * 4 + wave; i < r - 1; i += gridDim.x * 4) {
    const int64_t row = packed_slot(i, i + 1, b) - (i + 1);
    for (int j = i + 1 + lane; j < r; j += 64) {
      const float gv = g[row + j], mv = k.moment(m[row + j], gv);
      m[row + j] = mv;
      const float u = k.update(mv, gv);
      sum += (double)u * u;
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) red[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[(int64_t)z * gridDim.x + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// X planes of every block from its update, scaled by sx / (|M|_F + eps): one 64 x 64 tile on or above the
// diagonal per workgroup and, off the diagonal, its negated mirror; zeros from r to the padded size.
__global__ __launch_bounds__(256) void k_muon_unpack(MuonTable tab, int b, MuonK k, const double* __restrict__ part,
                                                     int parts, float sx, Planes X) {
  __shared__ float t[64][65];
  const int z = blockIdx.y;
  int s, r;
  int64_t off;
  tab.at(z, b, s, off, r);
  int ti, tj;
  upper_tile(blockIdx.x, (int)(X.ld / 64), ti, tj);
  const int i0 = ti * 64, j0 = tj * 64, live = (r + 127) / 128 * 128;
  if (j0 >= live) return;  // tiles that no product reads
  double ss = 0.0;
  for (int p = 0; p < parts; ++p) ss += part[(int64_t)z * parts + p];
  const double f = (double)sx / (__builtin_sqrt(2.0 * ss) + (double)k.eps);  // both halves of M
  const int c = threadIdx.x & 63, rr = threadIdx.x >> 6;
  const float* g = tab.g[s] + off;
  const float* m = tab.m[s] + off;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int i = i0 + rr + 4 * e, j = j0 + c;
    float v = 0.f;
    if (i < j && j < r) {
      const int64_t x = packed_slot(i, j, b);
      v = (float)((double)k.update(m[x], g[x]) * f);
    }
    t[rr + 4 * e][c] = v;
  }
  __syncthreads();
  const Planes o = X.at(z, 0);
  auto put = [&](int row0, int col0, auto value) {
#pragma unroll
    for (int w = threadIdx.x; w < 64 * 8; w += 256) {
      const int row = w / 8, col = w % 8 * 8;
      uint32_t h[4], l[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a = pack_hilo(value(row, col + 2 * e)), c2 = pack_hilo(value(row, col + 2 * e + 1));
        h[e] = (a & 0xffff) | (c2 << 16);
        l[e] = (a >> 16) | (c2 & 0xffff0000u);
      }
      const int64_t at = (row0 + row) * o.ld + col0 + col;
      *reinterpret_cast<uint4*>(o.h + at) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(o.l + at) = make_uint4(l[0], l[1], l[2], l[3]);
    }
  };
  if (ti == tj) {
    put(i0, j0, [&](int i, int j) { return i < j ? t[i][j] : i > j ? -t[j][i] : 0.f; });
  } else {
    put(i0, j0, [&](int i, int j) { return t[i][j]; });
    put(j0, i0, [&](int j, int i) { return -t[i][j]; });
  }
}

// One product of the batch on its tiles on and above the diagonal: out = alpha aux + beta a b^T, its mirror
// flipped by `flip`; with LAST the step of q instead of an output.
template <class C, bool AUX, bool LAST>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(2))) void k_ns_skew(MuonTable tab, int b, int tiles, Planes a, Planes bb, Planes aux,
                                                   Planes out, float alpha, float beta, uint32_t flip, MuonK k) {
  extern __shared__ __align__(16) unsigned char smem[];
  char* lds = reinterpret_cast<char*>(smem);
  const int per = tiles * (tiles + 1) / 2;
  const int u = xcd_unit(blockIdx.x, gridDim.x), z = u / per;
  int s, r, ti, tj;
  int64_t off;
  tab.at(z, b, s, off, r);
  upper_tile(u % per, tiles, ti, tj);
  const int m0 = ti * C::BM, n0 = tj * C::BN;
  if (n0 >= r) return;  // past the live corner: read by no product
  Acc<C> acc;
  ns_loop<C>(lds, a.at(z, m0), bb.at(z, n0), (r + C::BK - 1) / C::BK, ti == tj && a.h == bb.h, acc);
  const Planes none{};
  const Planes x = AUX ? aux.tile(z, m0, n0) : none;
  if constexpr (!LAST) {
    ns_store<C>(lds, acc, x, alpha, beta, out.tile(z, m0, n0), ti == tj ? none : out.tile(z, n0, m0), flip, nullptr);
  } else {
    float* q = tab.q[s] + off;
    const float sc = k.scale(r);
    ns_store<C>(lds, acc, x, alpha, beta, none, none, 0, [&](int r0, const float* st) {
#pragma unroll 4
      for (int c = threadIdx.x; c < C::RS * C::BN; c += C::NT) {
        const int i = c / C::BN, j = c % C::BN, row = m0 + r0 + i, col = n0 + j;
        if (row < col && col < r) {
          float* p = q + packed_slot(row, col, b);
          *p = k.step(*p, st[i * C::PITCH + j], sc);
        }
      }
    });
  }
}

// Blocks of b <= 128: one workgroup keeps X and A (then B) of its block in LDS
// for the whole step, from the momentum to the step of q, so that a call is one
// launch.  W waves share the P x P tile; a block of r < P runs its k-steps to r
// only, and waves whose part lies past r only keep the barriers.
template <int P, int W>
__global__ __launch_bounds__(W * 64) void k_muon_small(MuonTable tab, int b, MuonK k, int steps, float ca, float cb,
                                                       float cc, float sx) {
  constexpr int LD = P + 8, WN = W == 4 ? 2 : 1, TM = P / 32 / WN;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ double red[W];
  f16* Xh = reinterpret_cast<f16*>(smem);
  f16 *Xl = Xh + P * LD, *Ah = Xl + P * LD, *Al = Ah + P * LD;
  const int z = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s, r;
  int64_t off;
  tab.at(z, b, s, off, r);
  const float* g = tab.g[s] + off;
  float* m = tab.m[s] + off;
  float* q = tab.q[s] + off;
  double sum = 0.0;
  for (int i = wave; i < r - 1; i += W) {
    const int64_t row = packed_slot(i, i + 1, b) - (i + 1);
    for (int j = i + 1 + lane; j < r; j += 64) {
      const float gv = g[row + j], mv = k.moment(m[row + j], gv);
      m[row + j] = mv;
      const float u = k.update(mv, gv);
      sum += (double)u * u;
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) red[wave] = sum;
  // X planes start as zeros
  for (int c = threadIdx.x; c < 2 * P * LD / 8; c += W * 64) reinterpret_cast<uint4*>(Xh)[c] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  sum = red[0];
#pragma unroll
  for (int w = 1; w < W; ++w) sum += red[w];
  const double f = (double)sx / (__builtin_sqrt(2.0 * sum) + (double)k.eps);
  for (int i = wave; i < r - 1; i += W) {
    const int64_t row = packed_slot(i, i + 1, b) - (i + 1);
    for (int j = i + 1 + lane; j < r; j += 64) {  // the slots this thread wrote
      const float v = (float)((double)k.update(m[row + j], g[row + j]) * f);
      const f16 h = (f16)v, l = (f16)(v - (float)h);
      Xh[i * LD + j] = h;
      Xl[i * LD + j] = l;
      Xh[j * LD + i] = -h;
      Xl[j * LD + i] = -l;
    }
  }
  __syncthreads();
  const int m0 = wave / WN * TM * 32, n0 = wave % WN * TM * 32;
  const bool idle = m0 >= r || n0 >= r;
  const int ks_n = (r + 15) / 16, fr = lane & 31, fk = (lane >> 5) * 8;
  f32x16_v acc[TM][TM];
  auto product = [&](const f16* ah, const f16* al, const f16* bh, const f16* bl) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    if (idle) return;
    for (int ks = 0; ks < ks_n; ++ks) {
      f16x8_v fah[TM], fal[TM], fbh[TM], fbl[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int ra = (m0 + i * 32 + fr) * LD + ks * 16 + fk, rb = (n0 + i * 32 + fr) * LD + ks * 16 + fk;
        fah[i] = *reinterpret_cast<const f16x8_v*>(ah + ra);
        fal[i] = *reinterpret_cast<const f16x8_v*>(al + ra);
        fbh[i] = *reinterpret_cast<const f16x8_v*>(bh + rb);
        fbl[i] = *reinterpret_cast<const f16x8_v*>(bl + rb);
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fal[i], fbh[j], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fah[i], fbl[j], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fah[i], fbh[j], acc[i][j], 0, 0, 0);
        }
    }
  };
  // element = fn(row, col, element) over the wave's part
  auto each = [&](auto&& fn) __attribute__((always_inline)) {
    if (idle) return;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          acc[i][j][e] =
              fn(m0 + i * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3), n0 + j * 32 + (lane & 31), (float)acc[i][j][e]);
  };
  auto put = [&](f16* h, f16* l) __attribute__((always_inline)) {
    each([&](int row, int col, float v) {
      const f16 hv = (f16)v;
      h[row * LD + col] = hv;
      l[row * LD + col] = (f16)(v - (float)hv);
      return v;
    });
  };
  const float sc = k.scale(r);
  for (int it = 0; it < steps; ++it) {
    product(Xh, Xl, Xh, Xl);  // A = X X^T
    each([&](int, int, float v) { return v * (kSA / (sx * sx)); });
    put(Ah, Al);  // its readers of the last step are past the barrier
    __syncthreads();
    product(Ah, Al, Ah, Al);  // B = b A + c A A
    each([&](int row, int col, float v) {
      return cb * ((float)Ah[row * LD + col] + (float)Al[row * LD + col]) + cc / kSA * v;
    });
    __syncthreads();
    put(Ah, Al);
    __syncthreads();
    product(Ah, Al, Xh, Xl);  // a X - B X^T
    each([&](int row, int col, float v) {
      return ca * ((float)Xh[row * LD + col] + (float)Xl[row * LD + col]) - v / kSA;
    });
    if (it + 1 == steps) {
      each([&](int row, int col, float v) {
        if (row < col && col < r) {
          float* p = q + packed_slot(row, col, b);
          *p = k.step(*p, v / sx, sc);
        }
        return v;
      });
      return;
    }
    __syncthreads();
    put(Xh, Xl);
    __syncthreads();
  }
}

// -------------------------------------------------------- dense matrices ---

// A rows x cols matrix of the batch seen with its short side first: X[i][k] = G[i][k], or G[k][i] with `flip`.
template <typename T> struct Dense {
  T* p;
  int64_t ld, stride;
  int r, k, flip;
  PX_DEV T* at(int z, int64_t i, int64_t kk) const { return p + z * stride + (flip ? kk * ld + i : i * ld + kk); }
};

// each workgroup's sum of squares in 64 bits over rows blockIdx.x, + gridDim.x, ... of the stored matrix
template <typename T>
__global__ __launch_bounds__(256) void k_orth_norm(Dense<const T> G, double* __restrict__ part) {
  __shared__ double red[4];
  const int z = blockIdx.y, rows = G.flip ? G.k : G.r, cols = G.flip ? G.r : G.k;
  double sum = 0.0;
  for (int i = blockIdx.x; i < rows; i += gridDim.x) {
    const T* row = G.p + z * G.stride + i * G.ld;
    for (int j = threadIdx.x; j < cols; j += 256) {
      const double v = to_f32<T>(row[j]);
      sum += v * v;
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[(int64_t)z * gridDim.x + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// X and X^T planes from the matrix, scaled by sx / (|G|_F + eps), zeros past its ends: one 64 x 64 tile a workgroup.
template <typename T>
__global__ __launch_bounds__(256) void k_orth_load(Dense<const T> G, const double* __restrict__ part, int parts, float sx,
                                                   float eps, Planes X, Planes Xt) {
  __shared__ float t[64][65];
  const int z = blockIdx.y, tk = (int)(X.ld / 64), i0 = blockIdx.x / tk * 64, k0 = blockIdx.x % tk * 64;
  double ss = 0.0;
  for (int p = 0; p < parts; ++p) ss += part[(int64_t)z * parts + p];
  const double f = (double)sx / (__builtin_sqrt(ss) + (double)eps);
  const int c = threadIdx.x & 63, rr = threadIdx.x >> 6;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    // lanes run along the stored rows
    const int a = rr + 4 * e, i = i0 + (G.flip ? c : a), k = k0 + (G.flip ? a : c);
    t[i - i0][k - k0] = i < G.r && k < G.k ? (float)((double)to_f32<T>(*G.at(z, i, k)) * f) : 0.f;
  }
  __syncthreads();
  auto put = [&](const Planes& o, int row0, int col0, auto value) {
    for (int w = threadIdx.x; w < 64 * 8; w += 256) {
      const int row = w / 8, col = w % 8 * 8;
      uint32_t h[4], l[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a = pack_hilo(value(row, col + 2 * e)), b = pack_hilo(value(row, col + 2 * e + 1));
        h[e] = (a & 0xffff) | (b << 16);
        l[e] = (a >> 16) | (b & 0xffff0000u);
      }
      const int64_t at = (row0 + row) * o.ld + col0 + col;
      *reinterpret_cast<uint4*>(o.h + at) = make_uint4(h[0], h[1], h[2], h[3]);
      if (o.l) *reinterpret_cast<uint4*>(o.l + at) = make_uint4(l[0], l[1], l[2], l[3]);
    }
  };
  put(X.at(z, 0), i0, k0, [&](int i, int k) { return t[i][k]; });
  put(Xt.at(z, 0), k0, i0, [&](int k, int i) { return t[i][k]; });
}

template <class C>
PX_DEV void finish_sym(char* lds, const Acc<C>& acc, int z, int ti, int tj, const Planes& aux, const Planes& out,
                       float alpha, float beta) {
  const int m0 = ti * C::BM, n0 = tj * C::BN;
  const Planes none{};
  ns_store<C>(lds, acc, aux.tile(z, m0, n0), alpha, beta, out.tile(z, m0, n0), ti == tj ? none : out.tile(z, n0, m0), 0,
              nullptr);
}

// unit -> tile of a tm x tn grid, through groups of 8 row tiles, so that the workgroups that run together share
// both operands' panels
PX_DEV void x_tile(int id, int tm, int tn, int& bm, int& bn) {
  const int group = id / (8 * tn), first = group * 8, gs = min(tm - first, 8);
  bm = first + id % (8 * tn) % gs;
  bn = id % (8 * tn) / gs;
}

// Where the partial sums of a split product go: unit-major, then the accumulators in register order, 4 of them for
// every thread in turn, so that every access is 16 bytes a lane of whole lines.
template <class C> PX_DEV f32x4_v* part_at(float* part, int64_t unit, int i, int j, int g) {
  return reinterpret_cast<f32x4_v*>(part) + (((unit * C::TM + i) * C::TN + j) * 4 + g) * C::NT + threadIdx.x;
}

// out = alpha aux + beta a a^T, symmetric: its tiles on and above the diagonal.  With S > 1 splits of the K loop
// the workgroups write partial sums, which k_ns_join adds in order.
template <class C, bool SPLIT>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(2))) void k_ns_sym(int tiles, int KT, int S, Planes a, Planes aux, Planes out, float alpha,
                                                  float beta, float* __restrict__ part) {
  extern __shared__ __align__(16) unsigned char smem[];
  char* lds = reinterpret_cast<char*>(smem);
  const int per = tiles * (tiles + 1) / 2;
  const int u = xcd_unit(blockIdx.x, gridDim.x), z = u / (per * S), sp = u / per % S;
  int ti, tj;
  upper_tile(u % per, tiles, ti, tj);
  const int k0 = (int)((int64_t)sp * KT / S), k1 = (int)((int64_t)(sp + 1) * KT / S);
  Acc<C> acc;
  ns_loop<C>(lds, a.tile(z, ti * C::BM, k0 * C::BK), a.tile(z, tj * C::BN, k0 * C::BK), k1 - k0, C::BM == 128 && ti == tj,
             acc);  // (the 256 tile's registers leave no room for the second set of addresses)
  if constexpr (SPLIT) {
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *part_at<C>(part, u, i, j, g) = f32x4_v{acc.v[i][j][4 * g], acc.v[i][j][4 * g + 1], acc.v[i][j][4 * g + 2],
                                                  acc.v[i][j][4 * g + 3]};
  } else {
    finish_sym<C>(lds, acc, z, ti, tj, aux, out, alpha, beta);
  }
}

// the partial sums of one tile, in split order
template <class C>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(2))) void k_ns_join(int tiles, int S, Planes aux, Planes out, float alpha, float beta,
                                                   float* __restrict__ part) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int per = tiles * (tiles + 1) / 2, z = blockIdx.x / per, ut = blockIdx.x % per;
  int ti, tj;
  upper_tile(ut, tiles, ti, tj);
  Acc<C> acc;
  acc.zero();
  for (int sp = 0; sp < S; ++sp)
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4_v v = *part_at<C>(part, ((int64_t)z * S + sp) * per + ut, i, j, g);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc.v[i][j][4 * g + e] += v[e];
        }
  finish_sym<C>(reinterpret_cast<char*>(smem), acc, z, ti, tj, aux, out, alpha, beta);
}

// X <- alpha X + beta B X on every tile; X is updated in place (a tile is read by its own workgroup only) and its
// transpose written to the other of two buffers, for the other workgroups still read this one.
template <class C>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(2))) void k_ns_x(int tm, int tn, int KT, Planes B, Planes Xt, Planes X, Planes Xt_out,
                                                float alpha, float beta) {
  extern __shared__ __align__(16) unsigned char smem[];
  char* lds = reinterpret_cast<char*>(smem);
  const int u = xcd_unit(blockIdx.x, gridDim.x), z = u / (tm * tn);
  int bm, bn;
  x_tile(u % (tm * tn), tm, tn, bm, bn);
  const int m0 = bm * C::BM, n0 = bn * C::BN;
  Acc<C> acc;
  ns_loop<C>(lds, B.at(z, m0), Xt.at(z, n0), KT, false, acc);
  const Planes o = X.tile(z, m0, n0);
  ns_store<C>(lds, acc, o, alpha, beta, o, Xt_out.tile(z, n0, m0), 0, nullptr);
}

// The last step: alpha X + beta B X to the caller's matrix.
template <class C, typename T>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(2))) void k_ns_out(int tm, int tn, int KT, Planes B, Planes Xt, Planes X, Dense<T> O,
                                                  float alpha, float beta) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int u = xcd_unit(blockIdx.x, gridDim.x), z = u / (tm * tn);
  int bm, bn;
  x_tile(u % (tm * tn), tm, tn, bm, bn);
  const int m0 = bm * C::BM, n0 = bn * C::BN;
  Acc<C> acc;
  ns_loop<C>(reinterpret_cast<char*>(smem), B.at(z, m0), Xt.at(z, n0), KT, false, acc);
  const Planes none{};
  ns_store<C>(reinterpret_cast<char*>(smem), acc, X.tile(z, m0, n0), alpha, beta, none, none, 0,
              [&](int r0, const float* st) {
    // lanes run along the stored rows
#pragma unroll 4
    for (int c = threadIdx.x; c < C::RS * C::BN; c += C::NT) {
      const int i = O.flip ? c % C::RS : c / C::BN, j = O.flip ? c / C::RS : c % C::BN;
      const int row = m0 + r0 + i, col = n0 + j;
      if (row < O.r && col < O.k) *O.at(z, row, col) = from_f32<T>(st[i * C::PITCH + j]);
    }
  });
}

constexpr int kNormParts = 256;  // workgroups (and 64-bit partial sums) of one matrix's norm

inline float pow2_near(double x) { return (float)std::exp2(std::round(std::log2(x))); }

}  // namespace

namespace pxk {

namespace {

size_t al256(size_t x) { return (x + 255) / 256 * 256; }

// Bump allocation; a null base only counts.
struct Carve {
  char* base;
  size_t off = 0;
  template <typename T> T* take(size_t n) {
    T* p = reinterpret_cast<T*>(base ? base + off : nullptr);
    off += al256(n * sizeof(T));
    return p;
  }
  Planes planes(int count, int64_t rows, int64_t ld, bool lo) {
    Planes p;
    p.ld = ld;
    p.stride = rows * ld;
    p.h = take<f16>((size_t)count * p.stride);
    p.l = lo ? take<f16>((size_t)count * p.stride) : nullptr;
    return p;
  }
};

struct MuonWs {
  double* part;
  Planes buf[3];
};
constexpr int kMomentumParts = 8;
MuonWs muon_plan(Carve& c, int blocks, int b) {
  MuonWs w{};
  if (b <= 128) return w;
  const int P = (int)round_up(b, 128);
  w.part = c.take<double>((size_t)blocks * kMomentumParts);
  for (Planes& p : w.buf) p = c.planes(blocks, P, P, true);
  return w;
}

template <int P, int W> hipError_t muon_small(const MuonTable& t, int b, const MuonK& k, const NsHyper& n, hipStream_t s) {
  constexpr int lds = 4 * P * (P + 8) * 2;
  const hipError_t e = allow_lds(k_muon_small<P, W>, lds);
  if (e != hipSuccess) return e;
  k_muon_small<P, W><<<t.first[t.count], W * 64, lds, s>>>(t, b, k, n.steps, (float)n.a, (float)n.b, (float)n.c,
                                                           8.f * pow2_near(std::sqrt((double)b)));
  return hipGetLastError();
}

}  // namespace

size_t muon_ws_bytes(int64_t blocks, int b) {
  Carve c{nullptr};
  muon_plan(c, (int)blocks, b);
  return c.off;
}

hipError_t muon_batch(int count, float* const* q, const float* const* g, float* const* m, const int* d, int b,
                      const MuonHyper& hp, void* ws, hipStream_t s) {
  if (count < 1 || count > kMaxSides) return hipErrorInvalidValue;
  MuonTable t{};
  t.count = count;
  for (int i = 0; i < count; ++i) {
    t.q[i] = q[i];
    t.g[i] = g[i];
    t.m[i] = m[i];
    t.d[i] = d[i];
    t.first[i + 1] = t.first[i] + nblocks(d[i], b);
  }
  const NsHyper& n = hp.ns;
  MuonK k{(float)hp.lr, (float)hp.weight_decay, (float)hp.beta, (float)(1.0 - hp.beta), (float)n.rms, (float)n.eps,
          hp.nesterov};
  if (b <= 32) return muon_small<32, 1>(t, b, k, n, s);
  if (b <= 64) return muon_small<64, 4>(t, b, k, n, s);
  if (b <= 128) return muon_small<128, 4>(t, b, k, n, s);
  using C = NSmall<3>;
  const int NB = t.first[count], P = (int)round_up(b, 128), tiles = P / C::BM;
  Carve c{reinterpret_cast<char*>(ws)};
  MuonWs w = muon_plan(c, NB, b);
  hipError_t e = allow_lds(k_ns_skew<C, false, false>, C::LDS);
  if (e == hipSuccess) e = allow_lds(k_ns_skew<C, true, false>, C::LDS);
  if (e == hipSuccess) e = allow_lds(k_ns_skew<C, true, true>, C::LDS);
  if (e != hipSuccess) return e;
  const float sx = 8.f * pow2_near(std::sqrt((double)b)), a = (float)n.a, bb = (float)n.b, cc = (float)n.c;
  k_muon_momentum<<<dim3(kMomentumParts, NB), 256, 0, s>>>(t, b, k, w.part);
  const unsigned t64 = (unsigned)(P / 64);
  k_muon_unpack<<<dim3(t64 * (t64 + 1) / 2, NB), 256, 0, s>>>(t, b, k, w.part, kMomentumParts, sx, w.buf[0]);
  const unsigned grid = (unsigned)(tiles * (tiles + 1) / 2) * NB;
  Planes X = w.buf[0], A = w.buf[1];
  const Planes B = w.buf[2];
  for (int it = 0; it < n.steps; ++it) {
    k_ns_skew<C, false, false><<<grid, C::NT, C::LDS, s>>>(t, b, tiles, X, X, X, A, 0.f, kSA / (sx * sx), 0, k);
    k_ns_skew<C, true, false><<<grid, C::NT, C::LDS, s>>>(t, b, tiles, A, A, A, B, bb, cc / kSA, 0, k);
    if (it + 1 < n.steps) {
      // X' over A, which no product reads any more
      k_ns_skew<C, true, false><<<grid, C::NT, C::LDS, s>>>(t, b, tiles, B, X, X, A, a, -1.f / kSA, 0x8000u, k);
      std::swap(X, A);
    } else {
      k_ns_skew<C, true, true><<<grid, C::NT, C::LDS, s>>>(t, b, tiles, B, X, X, A, a / sx, -1.f / (kSA * sx), 0, k);
    }
  }
  return hipGetLastError();
}

namespace {

struct OrthPlan {
  int r, k, np, tile, rp, kp, splits;
  double* part;
  float* sums;
  Planes X, Xt[2], A, B;
};

// The tile, the products per product and the split of the A product's K loop.
OrthPlan orth_plan(Carve& c, int count, int rows, int cols, int dt) {
  OrthPlan p{};
  p.r = std::min(rows, cols);
  p.k = std::max(rows, cols);
  // a short side of up to 128 leaves so few roundings to average over that fp16 products alone lose digits
  p.np = dt == F32 || p.r <= 128 ? 3 : 1;
  p.tile = (int64_t)count * cdiv(p.r, 256) * cdiv(p.k, 256) >= 256 ? 256 : 128;
  p.rp = (int)round_up(p.r, p.tile);
  p.kp = (int)round_up(p.k, p.tile);
  const int64_t tiles = p.rp / p.tile, units = tiles * (tiles + 1) / 2 * count;
  const int KT = (int)cdiv(p.k, p.np == 3 ? 32 : 64), slots = p.tile == 256 ? 256 : 512;
  p.splits = 1;
  double best = 0;
  for (int S = 1; S <= 32 && S * 4 <= KT; ++S) {
    // rounds of workgroups times the K tiles of one, and what S partial sums of every tile cost in K tiles
    const double cost = (double)cdiv(units * S, slots) * cdiv(KT, S) + (S > 1 ? 2.0 + 2.0 * S * units / slots : 0.0);
    if (S == 1 || cost < best) {
      p.splits = S;
      best = cost;
    }
  }
  const bool lo = p.np == 3;
  p.part = c.take<double>((size_t)count * kNormParts);
  p.X = c.planes(count, p.rp, p.kp, true);
  for (Planes& t : p.Xt) t = c.planes(count, p.kp, p.rp, lo);
  p.A = c.planes(count, p.rp, p.rp, lo);
  p.B = c.planes(count, p.rp, p.rp, lo);
  p.sums = p.splits > 1 ? c.take<float>((size_t)p.splits * units * p.tile * p.tile) : nullptr;
  return p;
}

template <class C, typename T>
hipError_t orth_run(const OrthPlan& p, int count, const Dense<const T>& G, const Dense<T>& O, const NsHyper& n,
                    hipStream_t s) {
  hipError_t e = allow_lds(k_ns_sym<C, false>, C::LDS);
  if (e == hipSuccess) e = allow_lds(k_ns_sym<C, true>, C::LDS);
  if (e == hipSuccess) e = allow_lds(k_ns_join<C>, C::EPI);
  if (e == hipSuccess) e = allow_lds(k_ns_x<C>, C::LDS);
  if (e == hipSuccess) e = allow_lds(k_ns_out<C, T>, C::LDS);
  if (e != hipSuccess) return e;
  const float sx = 8.f * pow2_near(std::sqrt((double)p.k)), a = (float)n.a, b = (float)n.b, c = (float)n.c;
  const float scale = n.rms > 0 ? (float)(n.rms * std::sqrt((double)p.k)) : 1.f;
  const int tm = p.rp / C::BM, tn = p.kp / C::BN, KT = (int)cdiv(p.k, C::BK), KR = (int)cdiv(p.r, C::BK);
  const unsigned sym = (unsigned)(tm * (tm + 1) / 2) * count, full = (unsigned)(tm * tn) * count;
  const Planes none{};
  k_orth_norm<T><<<dim3(kNormParts, count), 256, 0, s>>>(G, p.part);
  k_orth_load<T><<<dim3((unsigned)(p.rp / 64) * (p.kp / 64), count), 256, 0, s>>>(G, p.part, kNormParts, sx, (float)n.eps,
                                                                              p.X, p.Xt[0]);
  for (int it = 0; it < n.steps; ++it) {
    const Planes &cur = p.Xt[it & 1], &nxt = p.Xt[(it + 1) & 1];
    if (p.splits > 1)
      k_ns_sym<C, true><<<sym * p.splits, C::NT, C::LDS, s>>>(tm, KT, p.splits, p.X, none, p.A, 0.f, kSA / (sx * sx), p.sums);
    else
      k_ns_sym<C, false><<<sym, C::NT, C::LDS, s>>>(tm, KT, 1, p.X, none, p.A, 0.f, kSA / (sx * sx), nullptr);
    if (p.splits > 1)
      k_ns_join<C><<<sym, C::NT, C::EPI, s>>>(tm, p.splits, none, p.A, 0.f, kSA / (sx * sx), p.sums);
    k_ns_sym<C, false><<<sym, C::NT, C::LDS, s>>>(tm, KR, 1, p.A, p.A, p.B, b, c / kSA, nullptr);
    if (it + 1 < n.steps)
      k_ns_x<C><<<full, C::NT, C::LDS, s>>>(tm, tn, KR, p.B, cur, p.X, nxt, a, 1.f / kSA);
    else
      k_ns_out<C, T><<<full, C::NT, C::LDS, s>>>(tm, tn, KR, p.B, cur, p.X, O, a * scale / sx, scale / (kSA * sx));
  }
  return hipGetLastError();
}

template <typename T>
hipError_t orth_t(int count, int rows, int cols, int dt, const void* G, int64_t ldg, int64_t sg, void* O, int64_t ldo,
                  int64_t so, const NsHyper& n, void* ws, hipStream_t s) {
  Carve c{reinterpret_cast<char*>(ws)};
  const OrthPlan p = orth_plan(c, count, rows, cols, dt);
  const int flip = rows > cols;
  const Dense<const T> g{reinterpret_cast<const T*>(G), ldg, sg, p.r, p.k, flip};
  const Dense<T> o{reinterpret_cast<T*>(O), ldo, so, p.r, p.k, flip};
  if (p.tile == 256)
    return p.np == 3 ? orth_run<NBig<3>, T>(p, count, g, o, n, s) : orth_run<NBig<1>, T>(p, count, g, o, n, s);
  return p.np == 3 ? orth_run<NSmall<3>, T>(p, count, g, o, n, s) : orth_run<NSmall<1>, T>(p, count, g, o, n, s);
}

}  // namespace

size_t orth_ws_bytes(int count, int rows, int cols, int dt) {
  Carve c{nullptr};
  orth_plan(c, count, rows, cols, dt);
  return c.off;
}

hipError_t orthogonalize(int count, int rows, int cols, int dt, const void* G, int64_t ldg, int64_t sg, void* O,
                         int64_t ldo, int64_t so, const NsHyper& n, void* ws, hipStream_t s) {
  if (dt == BF16) return orth_t<bf16_t>(count, rows, cols, dt, G, ldg, sg, O, ldo, so, n, ws, s);
  return orth_t<float>(count, rows, cols, dt, G, ldg, sg, O, ldo, so, n, ws, s);
}

}  // namespace pxk
