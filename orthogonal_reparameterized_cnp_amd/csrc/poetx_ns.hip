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
// of two: hi = fp16(x), lo = fp16(2^11 (x - hi)), together x to 2^-23 of itself
// down to 2^-14 and to 2^-36 below (a lo of x - hi itself would lose digits from
// 2^-3 down, where it is subnormal: rows at 1e-3 of the others came out 1e-4 of
// themselves off, a matrix with a row 1e4 times the others 2e-5 of its norm).
// The products run on the fp16 matrix instructions with fp32 accumulation, hi hi
// + 2^-11 (hi lo + lo hi), the two sums in accumulators of their own: as exact
// as fp32 products (the low-by-low part is 2^-22 of the whole) at three times
// the cost of one, about 5x the rate of the fp32 matrix instructions.
// bf16 matrices take the same products and are rounded once, at the end.  (hi hi
// alone is 2.5 times as fast, but its roundings of 2^-12 pass through all steps:
// a matrix of low rank and noise comes out 1.2 to 2.4e-3 of its norm off, a
// diagonal of four entries, where nothing averages them, 1.3e-2.)
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
#include <atomic>
#include <cmath>
#include <cstddef>

#include "kernel_util.h"

using namespace px;

namespace {

typedef _Float16 f16;
typedef _Float16 f16x8_v __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4_v __attribute__((ext_vector_type(4)));

constexpr float kSA = 256.f;  // scale of A and B
constexpr int kInter = 32;    // run of hi values between runs of lo values
constexpr float kLo = 2048.f;  // scale of the lo values

// Tile configuration of the product kernels: two planes per operand, a ring of S stages of BK columns.
template <int BM_, int BN_, int BK_, int WM_, int WN_, int S_> struct NCfg {
  static constexpr int BM = BM_, BN = BN_, BK = BK_, WM = WM_, WN = WN_, STAGES = S_;
  static constexpr int NW = WM * WN, NT = NW * 64;
  static constexpr int WTM = BM / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
  static constexpr int A_BYTES = 2 * BM * BK * 2, B_BYTES = 2 * BN * BK * 2;  // one stage
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int LA = A_BYTES / 1024 / NW, LB = B_BYTES / 1024 / NW;  // copies per wave and stage
  // the epilogue stages the tile as (hi, lo) words; a pitch of 5 mod 64 words spreads both the reads along its rows
  // and those down its columns over the banks
  static constexpr int PITCH = BN + 5, EPI = BM * PITCH * 4;
  static constexpr int LDS = S_ * STAGE > EPI ? S_ * STAGE : EPI;
  static_assert(A_BYTES % (1024 * NW) == 0 && B_BYTES % (1024 * NW) == 0, "tile must split into 1 KB per wave");
  // the K loops run to the next multiple of BK past the last column: no further than the tiles of 64 that hold it
  static_assert(64 % BK == 0, "K steps stay within written tiles");
  static_assert(BM == BN && PITCH % 64 == 5, "epilogue stage");
};
// 4 waves of 32 x 32, two workgroups a CU: products too small to fill the GPU with larger tiles, bound by latency (two
// stages of 64 columns have half the barriers of four of 32, which took 4 % longer on 40 blocks of 256)
using NTiny = NCfg<64, 64, 64, 2, 2, 2>;
// 4 waves of 64 x 64, two workgroups a CU
using NSmall = NCfg<128, 128, 32, 2, 2, 2>;

PX_DEV f16x8_v as_f16(const bf16x8_v& x) {
  f16x8_v y;
  __builtin_memcpy(&y, &x, 16);
  return y;
}

PX_DEV f16 low_half(float v, f16 h) { return (f16)((v - (float)h) * kLo); }

PX_DEV uint32_t pack_hilo(float v) {
  const f16 h = (f16)v, l = low_half(v, h);
  uint16_t hb, lb;
  __builtin_memcpy(&hb, &h, 2);
  __builtin_memcpy(&lb, &l, 2);
  return (uint32_t)hb | ((uint32_t)lb << 16);
}

// One operand: K-contiguous rows, ld fp16 elements apart, in which kInter hi values and then their lo values alternate,
// so that a K step of 32 is one 128-byte line of every row.
struct Planes {
  f16* h = nullptr;
  int64_t ld = 0, stride = 0;  // stride: fp16 elements from one matrix of the batch to the next
  // the planes from (row, col) of matrix z on; col a multiple of 32
  PX_DEV Planes tile(int z, int64_t row, int64_t col) const {
    if (!h) return *this;
    return Planes{h + z * stride + row * ld + 2 * col, ld, stride};
  }
};
// place of a row's hi value from its planes' origin; its lo value is kInter further
PX_DEV constexpr int plane_col(int j) { return j / kInter * 2 * kInter + j % kInter; }

// acc = sum over KT tiles of K of a's tile rows times b's tile rows.  `same`: the two tiles are one.  `upper`: only
// what lies on and above the tile's diagonal is wanted, so that waves whose part lies below it multiply nothing (and
// results do not depend on the tile a block ran on: what is below a diagonal is always a mirror).
template <class C>
PX_DEV void ns_loop(char* lds, const Planes& a, const Planes& b, int KT, bool same, Acc<C>& acc, bool upper = false) {
  constexpr int PK = C::BK * 2;  // fp16 elements of a row in a stage
  const AccPos<C> p = acc_pos<C>();
  const int wave = threadIdx.x >> 6, lane = p.lane;
  auto issue = [&](int kt, char* st) {
    dma_kmaj<C::BM, PK, C::NW>(reinterpret_cast<const bf16_t*>(a.h), a.ld, kt * PK, st, wave, lane);
    if (same) return;
    dma_kmaj<C::BN, PK, C::NW>(reinterpret_cast<const bf16_t*>(b.h), b.ld, kt * PK, st + C::A_BYTES, wave, lane);
  };
  Acc<C> cross;  // kLo times the products of hi and lo values
  acc.zero();
  cross.zero();
#pragma unroll
  for (int t = 0; t < C::STAGES - 1; ++t)
    if (t < KT) issue(t, lds + t * C::STAGE);
  struct Frags {
    f16x8_v ah[C::TM], bh[C::TN], al[C::TM], bl[C::TN];
  };
  for (int kt = 0; kt < KT; ++kt) {
    // the copies of up to STAGES - 2 later stages may stay in flight; stage kt must have landed
    if (C::STAGES == 2 || KT - 1 - kt < C::STAGES - 2)
      wait_vm<0>();
    else if (same)
      wait_vm<(C::STAGES - 2) * C::LA>();
    else
      wait_vm<(C::STAGES - 2) * (C::LA + C::LB)>();
    wait_lgkm0();
    barrier_raw();
    const int nxt = kt + C::STAGES - 1;
    if (nxt < KT) issue(nxt, lds + nxt % C::STAGES * C::STAGE);
    if (upper && p.wm > p.wn) continue;
    const char* As = lds + kt % C::STAGES * C::STAGE;
    const char* Bs = same ? As : As + C::A_BYTES;
    // place of k-step ks's hi values in a staged row
    auto hi = [](int ks) { return plane_col(ks * 16); };
    auto load = [&](int ks, Frags& f) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < C::TM; ++i) {
        const int t0 = p.wm * C::WTM + i * 32;
        f.ah[i] = as_f16(frag_kmaj<PK>(As, t0, hi(ks), lane));
        f.al[i] = as_f16(frag_kmaj<PK>(As, t0, hi(ks) + kInter, lane));
      }
#pragma unroll
      for (int j = 0; j < C::TN; ++j) {
        const int t0 = p.wn * C::WTN + j * 32;
        f.bh[j] = as_f16(frag_kmaj<PK>(Bs, t0, hi(ks), lane));
        f.bl[j] = as_f16(frag_kmaj<PK>(Bs, t0, hi(ks) + kInter, lane));
      }
    };
    constexpr int KS = C::BK / 16;
    Frags f[2];
    load(0, f[0]);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Frags& c = f[ks & 1];
      if (ks + 1 < KS) load(ks + 1, f[(ks + 1) & 1]);
#pragma unroll
      for (int i = 0; i < C::TM; ++i)
#pragma unroll
        for (int j = 0; j < C::TN; ++j) {
          cross.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(c.al[i], c.bh[j], cross.v[i][j], 0, 0, 0);
          cross.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(c.ah[i], c.bl[j], cross.v[i][j], 0, 0, 0);
          acc.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(c.ah[i], c.bh[j], acc.v[i][j], 0, 0, 0);
        }
      // ask the compiler to interleave the reads with the matrix instructions
      __builtin_amdgcn_iglp_opt(1);
    }
  }
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < C::TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc.v[i][j][e] += cross.v[i][j][e] * (1.f / kLo);
  wait_lgkm0();
  barrier_raw();
}

PX_DEV float plane_value(f16 h, f16 l) { return (float)h + (float)l * (1.f / kLo); }

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

typedef uint32_t u32x4_v __attribute__((ext_vector_type(4)));
// 16 bytes to memory.  Small products (NT) write past the L2: what they leave dirty there is written back after their
// last wave, before the next launch may start (it took a step of 40 blocks of 256 from 153 to 144 us; one of 160 blocks
// of 512, whose write-back runs under other tiles, would go from 1882 to 1926).
template <bool NT> PX_DEV void put16(f16* p, const uint4& v) {
  if constexpr (NT)
    __builtin_nontemporal_store(u32x4_v{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4_v*>(p));
  else
    *reinterpret_cast<uint4*>(p) = v;
}

// The epilogue of a tile, v = alpha aux + beta acc, through LDS: the accumulators are staged in fp32, then each thread
// takes 8 consecutive values of a row, adds the aux planes' (16-byte loads; null: none), writes them to the planes `o`
// (null: none) and leaves them in LDS, as (hi, lo) words where `t` (the transposed tile's planes; null: none) is
// written from there with `flip` (0x8000 negates), as floats for emit(stage).  All planes are at the tile's origin.
// `diag` (with `t` the tile itself): the tile lies on the diagonal of a symmetric or, with `flip`, skew matrix, and its
// values below the diagonal are the mirrors of those above.  A computed skew matrix would be off by its roundings
// there, and the products that read X^T as -X, from rows alone, would see the sign of that symmetric part turned over:
// it grows by about 5 a step where a rounding otherwise grows by 3.4.
template <class C, class Emit>
PX_DEV void ns_store(char* lds, const Acc<C>& acc, const Planes& aux, float alpha, float beta, const Planes& o,
                     const Planes& t, uint32_t flip, const Emit& emit, bool diag = false) {
  constexpr bool EMIT = !std::is_same<Emit, std::nullptr_t>::value;
  constexpr int NIT = C::BM * C::BN / 8 / C::NT;  // a thread's share of the pieces of 8
  static_assert(C::BM * C::BN / 8 % C::NT == 0, "whole shares");
  uint32_t* st = reinterpret_cast<uint32_t*>(lds);
  const AccPos<C> p = acc_pos<C>();
  // the aux values: a thread's whole share is on its way before the stage is written
  f16x8_v xh[NIT], xl[NIT];
  if (aux.h) {
#pragma unroll
    for (int x = 0; x < NIT; ++x) {
      const int c = threadIdx.x + x * C::NT, i = c / (C::BN / 8), j = c % (C::BN / 8) * 8;
      const int64_t at = i * aux.ld + plane_col(j);
      xh[x] = *reinterpret_cast<const f16x8_v*>(aux.h + at);
      xl[x] = *reinterpret_cast<const f16x8_v*>(aux.h + at + kInter);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < C::TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) st[p.row(i, e) * C::PITCH + p.col(j)] = __float_as_uint(beta * acc.v[i][j][e]);
  __syncthreads();
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    const int c = threadIdx.x + it * C::NT, i = c / (C::BN / 8), j = c % (C::BN / 8) * 8;
    uint32_t* w = st + i * C::PITCH + j;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
    if (aux.h) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += alpha * plane_value(xh[it][e], xl[it][e]);
    }
    if constexpr (EMIT) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(v[e]);
    } else {
      uint32_t x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = pack_hilo(v[e]);
      if (!diag) {
        uint4 h, l;
        split_words(x, 0, h, l);
        const int64_t at = i * o.ld + plane_col(j);
        put16<C::BM == 64>(o.h + at, h);
        put16<C::BM == 64>(o.h + at + kInter, l);
      }
      if (t.h || diag)
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = x[e];
    }
  }
  if constexpr (EMIT) {
    __syncthreads();
    emit(reinterpret_cast<const float*>(st));
  } else if (diag) {
    __syncthreads();
#pragma unroll 2
    for (int c = threadIdx.x; c < C::BM * C::BN / 8; c += C::NT) {
      const int i = c / (C::BN / 8), j = c % (C::BN / 8) * 8;
      uint32_t x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t up = st[min(i, j + e) * C::PITCH + max(i, j + e)];
        x[e] = j + e > i ? up : j + e < i ? up ^ (flip | flip << 16) : flip ? 0u : up;
      }
      uint4 h, l;
      split_words(x, 0, h, l);
      const int64_t at = i * o.ld + plane_col(j);
      put16<C::BM == 64>(o.h + at, h);
      put16<C::BM == 64>(o.h + at + kInter, l);
    }
  } else if (t.h) {
    __syncthreads();
#pragma unroll 2
    for (int c = threadIdx.x; c < C::BM * C::BN / 8; c += C::NT) {
      const int j = c / (C::BM / 8), i = c % (C::BM / 8) * 8;
      uint32_t x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = st[(i + e) * C::PITCH + j];
      uint4 h, l;
      split_words(x, flip | (flip << 16), h, l);
      const int64_t at = j * t.ld + plane_col(i);
      put16<C::BM == 64>(t.h + at, h);
      put16<C::BM == 64>(t.h + at + kInter, l);
    }
  }
}

// one 64 x 64 tile of floats, value(row, col), to matrix z's planes at (row0, col0); 256 threads
template <class F> PX_DEV void put64(const Planes& p, int z, int64_t row0, int64_t col0, const F& value) {
  const Planes o = p.tile(z, row0, col0);
#pragma unroll
  for (int w = threadIdx.x; w < 64 * 8; w += 256) {
    const int row = w / 8, col = w % 8 * 8;
    uint32_t x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = pack_hilo(value(row, col + e));
    uint4 h, l;
    split_words(x, 0, h, l);
    const int64_t at = row * o.ld + plane_col(col);
    *reinterpret_cast<uint4*>(o.h + at) = h;
    *reinterpret_cast<uint4*>(o.h + at + kInter) = l;
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
  int z0;  // number of the launch's first block
  // block z of the launch: its side, the first packed slot of it in the side's arrays, its live size
  PX_DEV void at(int z, int b, int& s, int64_t& off, int& r) const {
    z += z0;
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

// Row and column of a packed slot (b <= 1024): row i starts at slot i b - i (i + 1) / 2; the root's rounding is put
// right by at most a step.
PX_DEV int slot_start(int i, int b) { return i * b - i * (i + 1) / 2; }
PX_DEV int slot_i(int x, int b) {
  const float t = (float)(2 * b - 1);
  int i = (int)((t - __builtin_sqrtf(fmaxf(t * t - 8.f * (float)x, 0.f))) * 0.5f);
  i = max(0, min(i, b - 2));
  while (i > 0 && slot_start(i, b) > x) --i;
  while (slot_start(i + 1, b) <= x) ++i;
  return i;
}
PX_DEV int slot_j(int x, int b) {
  const int i = slot_i(x, b);
  return x - slot_start(i, b) + i + 1;
}

// What the products need of a block of the launch, in the workspace.
struct BlockInfo {
  float* q;  // its packed parameters
  int r;     // its live size
};

// Momentum of every live slot, and each workgroup's sum of the squared updates in 64 bits: workgroup c of block z
// takes the packed slots from 2048 c on, 8 consecutive ones a thread (of any alignment).  A dead slot (j >= r of a
// partial block) is neither read nor written.  Bound by bytes: 160 blocks of 512, 251 MB in 41.9 us, 6.0 TB/s.
constexpr int kMomentumSlots = 2048;
__global__ __launch_bounds__(256) void k_muon_momentum(MuonTable tab, int b, MuonK k, double* __restrict__ part,
                                                       BlockInfo* __restrict__ info) {
  __shared__ double red[4];
  const int z = blockIdx.y, slots = b * (b - 1) / 2;
  int s, r;
  int64_t off;
  tab.at(z, b, s, off, r);
  if (blockIdx.x == 0 && threadIdx.x == 0) info[z] = BlockInfo{tab.q[s] + off, r};
  const int x0 = blockIdx.x * kMomentumSlots + threadIdx.x * 8;
  const float* g = tab.g[s] + off + x0;
  float* m = tab.m[s] + off + x0;
  double sum = 0.0;
  if (r == b && x0 + 8 <= slots) {
    float gv[8], mv[8];
    __builtin_memcpy(gv, g, 32);
    __builtin_memcpy(mv, m, 32);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mv[e] = k.moment(mv[e], gv[e]);
      const float u = k.update(mv[e], gv[e]);
      sum += (double)u * u;
    }
    __builtin_memcpy(m, mv, 32);
  } else if (x0 < slots) {
    int i = slot_i(x0, b), j = x0 - slot_start(i, b) + i + 1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (x0 + e < slots && j < r) {
        const float mv = k.moment(m[e], g[e]), u = k.update(mv, g[e]);
        m[e] = mv;
        sum += (double)u * u;
      }
      if (++j == b) j = ++i + 1;
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[(int64_t)z * gridDim.x + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// the sum of n partial sums, the same in every wave of the grid
PX_DEV double sum_parts(const double* part, int n) {
  double s = 0.0;
  for (int p = threadIdx.x & 63; p < n; p += 64) s += part[p];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o);
  return s;
}

// X planes of every block from its update, scaled by sx / (|M|_F + eps): one 64 x 64 tile on or above the
// diagonal per workgroup and, off the diagonal, its negated mirror; zeros from r to the end of its last tile.
// 160 blocks of 512: 257 MB fetched (packed rows start anywhere in a line) and 168 MB written in 73 us, 5.8 TB/s.
__global__ __launch_bounds__(256) void k_muon_unpack(MuonTable tab, int b, MuonK k, const double* __restrict__ part,
                                                     int parts, float sx, int n64, Planes X) {
  __shared__ float t[64][65];
  const int z = blockIdx.y;
  int s, r;
  int64_t off;
  tab.at(z, b, s, off, r);
  int ti, tj;
  upper_tile(blockIdx.x, n64, ti, tj);
  const int i0 = ti * 64, j0 = tj * 64, live = (r + 127) / 128 * 128;
  if (j0 >= live) return;  // tiles that no product reads
  const int c = threadIdx.x & 63, rr = threadIdx.x >> 6;
  const float* g = tab.g[s] + off;
  const float* m = tab.m[s] + off;
  // dead and mirrored places read slot 0 (a live one wherever a block has any) in their stead, so that all loads are
  // under way together
  float gv[16], mv[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int i = i0 + rr + 4 * e, j = j0 + c;
    const int64_t x = i < j && j < r ? packed_slot(i, j, b) : 0;
    gv[e] = r > 1 ? g[x] : 0.f;
    mv[e] = r > 1 ? m[x] : 0.f;
  }
  const double f = (double)sx / (__builtin_sqrt(2.0 * sum_parts(part + (int64_t)z * parts, parts)) + (double)k.eps);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int i = i0 + rr + 4 * e, j = j0 + c;
    t[rr + 4 * e][c] = i < j && j < r ? (float)((double)k.update(mv[e], gv[e]) * f) : 0.f;  // (both halves of M: 2 sum)
  }
  __syncthreads();
  if (ti == tj) {
    put64(X, z, i0, j0, [&](int i, int j) { return i < j ? t[i][j] : i > j ? -t[j][i] : 0.f; });
  } else {
    put64(X, z, i0, j0, [&](int i, int j) { return t[i][j]; });
    put64(X, z, j0, i0, [&](int j, int i) { return -t[i][j]; });
  }
}

struct SkewArgs {
  Planes a, b, aux, out;
  float alpha, beta;
  uint32_t flip;
};

// One tile (ti, tj) of block z
template <class C, bool AUX, bool LAST>
PX_DEV void skew_tile(char* lds, const SkewArgs& g, const BlockInfo* info, int b, int z, int ti, int tj,
                      const MuonK& k) {
  const int r = info[z].r, m0 = ti * C::BM, n0 = tj * C::BN;
  if (n0 >= r) return;  // past the live corner: read by no product
  Acc<C> acc;
  ns_loop<C>(lds, g.a.tile(z, m0, 0), g.b.tile(z, n0, 0), (r + C::BK - 1) / C::BK, ti == tj && g.a.h == g.b.h, acc,
             ti == tj);
  const Planes none{};
  const Planes x = AUX ? g.aux.tile(z, m0, n0) : none;
  if constexpr (!LAST) {
    ns_store<C>(lds, acc, x, g.alpha, g.beta, g.out.tile(z, m0, n0), g.out.tile(z, n0, m0), g.flip, nullptr, ti == tj);
  } else {
    float* q = info[z].q;
    const float sc = k.scale(r);
    ns_store<C>(lds, acc, x, g.alpha, g.beta, none, none, 0, [&](const float* st) {
      // runs of 8 slots of a packed row (of any alignment)
#pragma unroll 2
      for (int c = threadIdx.x; c < C::BM * C::BN / 8; c += C::NT) {
        const int i = c / (C::BN / 8), j = c % (C::BN / 8) * 8, row = m0 + i, col = n0 + j;
        if (col + 7 <= row || col >= r) continue;
        float* p = q + packed_slot(row, col, b);
        const float* v = st + i * C::PITCH + j;
        if (col > row && col + 8 <= r) {
          float f[8];
          __builtin_memcpy(f, p, 32);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = k.step(f[e], v[e], sc);
          __builtin_memcpy(p, f, 32);
        } else {
          for (int e = 0; e < 8; ++e)
            if (col + e > row && col + e < r) p[e] = k.step(p[e], v[e], sc);
        }
      }
    });
  }
}

// One product of the batch on the tiles on and above the diagonal of its blocks: out = alpha aux + beta a b^T, its
// mirror flipped by `flip`; with LAST the step of q instead of an output.  The first `wide` blocks run on 128 x 128
// tiles, the rest, which would leave most of the last round of workgroups empty, on 64 x 64 ones.  160 blocks of 512:
// 113 us for A and 129 with the term of the planes, three rounds of workgroups, 715 and 625 TFLOP/s of the matrix
// instructions, which are busy 30 and 26 % of the time, while 0.36 and 0.49 GB pass the L2s (3.2 and 3.8 TB/s): a
// tile's copies, products and stores come in part one after the other; 40 blocks of 256: 8 to 9 us, bound by latency.
template <bool AUX, bool LAST>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void k_ns_skew(
    SkewArgs g, const BlockInfo* __restrict__ info, int b, int n128, int wide, MuonK k) {
  using C1 = NSmall;
  using C2 = NTiny;
  static_assert(C1::NT == 256 && C2::NT == 256, "one launch");
  extern __shared__ __align__(16) unsigned char smem[];
  char* lds = reinterpret_cast<char*>(smem);
  const int per1 = n128 * (n128 + 1) / 2, per2 = n128 * (2 * n128 + 1), units1 = wide * per1;
  int ti, tj;
  if ((int)blockIdx.x < units1) {
    const int u = xcd_unit(blockIdx.x, units1);
    upper_tile(u % per1, n128, ti, tj);
    skew_tile<C1, AUX, LAST>(lds, g, info, b, u / per1, ti, tj, k);
  } else {
    const int u = xcd_unit(blockIdx.x - units1, gridDim.x - units1);
    upper_tile(u % per2, 2 * n128, ti, tj);
    skew_tile<C2, AUX, LAST>(lds, g, info, b, wide + u / per2, ti, tj, k);
  }
}

// Blocks of b <= 128: one workgroup keeps X and A (then B) of its block in LDS
// for the whole step, from the momentum to the step of q, so that a call is one
// launch.  W waves share the P x P tile; a block of r < P runs its k-steps to r
// only, and waves whose part lies past r only keep the barriers.  Bound by latency: 16 blocks of 32 take 22.2 us, of
// which 15 dependent products about 0.75 us each.
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
  // the thread's slots threadIdx.x, + 64 W, ...: their places (i, j), packed, and their updates stay in registers
  // until the norm is known
  constexpr int NU = ((P * (P - 1) / 2 + W * 64 - 1) / (W * 64) + 7) / 8 * 8;
  const int slots = b * (b - 1) / 2;
  float u[NU];
  uint32_t ij[NU];
  double sum = 0.0;
  {
    int x = min((int)threadIdx.x, slots - 1), i = slot_i(x, b), j = x - slot_start(i, b) + i + 1;
    x = threadIdx.x;
#pragma unroll
    for (int e0 = 0; e0 < NU; e0 += 8) {
      float gv[8], mv[8];
#pragma unroll
      for (int e = 0; e < 8; ++e, x += W * 64) {
        const bool ok = x < slots && j < r;
        ij[e0 + e] = ok ? (uint32_t)(i << 16 | j) : 0u;  // (0, 0) is no slot's place
        gv[e] = ok ? g[x] : 0.f;
        mv[e] = ok ? m[x] : 0.f;
        j += W * 64;
        while (j >= b && i < b) j += ++i + 1 - b;  // the rows get shorter
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        mv[e] = k.moment(mv[e], gv[e]);
        if (ij[e0 + e]) m[(e0 + e) * W * 64 + threadIdx.x] = mv[e];
        u[e0 + e] = k.update(mv[e], gv[e]);
        sum += (double)u[e0 + e] * u[e0 + e];
      }
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) red[wave] = sum;
  // X planes start as zeros: the diagonal, and all past the live corner, stay so
  for (int c = threadIdx.x; c < 2 * P * LD / 8; c += W * 64) reinterpret_cast<uint4*>(Xh)[c] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  sum = red[0];
#pragma unroll
  for (int w = 1; w < W; ++w) sum += red[w];
  const double f = (double)sx / (__builtin_sqrt(2.0 * sum) + (double)k.eps);
#pragma unroll
  for (int e = 0; e < NU; ++e) {
    const int i = ij[e] >> 16, j = ij[e] & 0xffff;
    if (ij[e] == 0) continue;
    const float v = (float)((double)u[e] * f);
    const f16 h = (f16)v, l = low_half(v, h);
    Xh[i * LD + j] = h;
    Xl[i * LD + j] = l;
    Xh[j * LD + i] = -h;
    Xl[j * LD + i] = -l;
  }
  __syncthreads();
  const int m0 = wave / WN * TM * 32, n0 = wave % WN * TM * 32;
  const bool idle = m0 >= r || n0 >= r;
  const int ks_n = (r + 15) / 16, fr = lane & 31, fk = (lane >> 5) * 8;
  f32x16_v acc[TM][TM], cross[TM][TM];
  auto product = [&](const f16* ah, const f16* al, const f16* bh, const f16* bl) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = cross[i][j][e] = 0.f;
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
          cross[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fal[i], fbh[j], cross[i][j], 0, 0, 0);
          cross[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fah[i], fbl[j], cross[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fah[i], fbh[j], acc[i][j], 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] += cross[i][j][e] * (1.f / kLo);
  };
  // fn(row, col, values) over the wave's part in runs of 4 rows of one column, the unit a lane owns.  A and B are
  // symmetric and X is skew, so a run of a column is read and written as the run of the row col: 8 bytes, not 4 times 2
  auto each4 = [&](auto&& fn) __attribute__((always_inline)) {
    if (idle) return;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
          fn(m0 + i * 32 + 8 * q + 4 * (lane >> 5), n0 + j * 32 + (lane & 31), v);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] = v[e];
        }
  };
  auto put4 = [&](f16* h, f16* l, int at, const float (&v)[4]) __attribute__((always_inline)) {
    f16x4_v hv, lv;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      hv[e] = (f16)v[e];
      lv[e] = low_half(v[e], hv[e]);
    }
    *reinterpret_cast<f16x4_v*>(h + at) = hv;
    *reinterpret_cast<f16x4_v*>(l + at) = lv;
  };
  auto add4 = [&](const f16* h, const f16* l, int at, float f, float (&v)[4]) __attribute__((always_inline)) {
    const f16x4_v hv = *reinterpret_cast<const f16x4_v*>(h + at), lv = *reinterpret_cast<const f16x4_v*>(l + at);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += f * plane_value(hv[e], lv[e]);
  };
  const float sc = k.scale(r);
  for (int it = 0; it < steps; ++it) {
    product(Xh, Xl, Xh, Xl);  // A = X X^T; its place's readers of the last step are past the barrier
    each4([&](int row, int col, float(&v)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= kSA / (sx * sx);
      put4(Ah, Al, col * LD + row, v);
    });
    __syncthreads();
    product(Ah, Al, Ah, Al);  // B = b A + c A A
    each4([&](int row, int col, float(&v)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= cc / kSA;
      add4(Ah, Al, col * LD + row, cb, v);
    });
    __syncthreads();
    each4([&](int row, int col, float(&v)[4]) { put4(Ah, Al, col * LD + row, v); });
    __syncthreads();
    product(Ah, Al, Xh, Xl);  // a X - B X^T, with X[row][col] read as -X[col][row]
    each4([&](int row, int col, float(&v)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= -1.f / kSA;
      add4(Xh, Xl, col * LD + row, -ca, v);
    });
    if (it + 1 == steps) {
      each4([&](int row, int col, float(&v)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (row + e < col && col < r) {
            float* p = q + packed_slot(row + e, col, b);
            *p = k.step(*p, v[e] / sx, sc);
          }
      });
      return;
    }
    __syncthreads();
    // X stays exactly skew (see ns_store): its upper half, and the negated mirror
    each4([&](int row, int col, float(&v)[4]) {
      if (row >= col) return;
      const float n[4] = {-v[0], -v[1], -v[2], -v[3]};
      if (row + 3 < col) put4(Xh, Xl, col * LD + row, n);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (row + e < col) {
          const f16 hv = (f16)v[e], lv = low_half(v[e], hv);
          Xh[(row + e) * LD + col] = hv;
          Xl[(row + e) * LD + col] = lv;
          if (row + 3 >= col) {
            Xh[col * LD + row + e] = -hv;
            Xl[col * LD + row + e] = -lv;
          }
        }
    });
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

// 8 elements from c of a stored row of n, zeros past its end; rows need no alignment beyond the element's
template <typename T> struct Run8 {
  static constexpr int N = sizeof(T) / 2;
  u32x4_v v[N];
  PX_DEV void load(const T* row, int64_t c, int64_t n) {
    if (c + 8 <= n) {
      __builtin_memcpy(v, row + c, sizeof(v));
    } else {
      T t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = c + e < n ? row[c + e] : T(0);
      __builtin_memcpy(v, t, sizeof(v));
    }
  }
  PX_DEV void get(float (&f)[8]) const {
    // the compiler would take 16-bit elements apart where they are loaded, and wait for every load there
    u32x4_v w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[i] = v[i];
      asm volatile("" : "+v"(w[i]));
    }
    T t[8];
    __builtin_memcpy(t, w, sizeof(v));
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = to_f32<T>(t[e]);
  }
};

// each workgroup's sum of squares in 64 bits: the runs of 8 elements of the stored rows, dealt to the grid's threads,
// four of them under way at a time (4096 x 14336 bf16: 117 MB in 24.1 us, 4.9 TB/s; eight at a time 28.1)
template <typename T>
__global__ __launch_bounds__(256) void k_orth_norm(Dense<const T> G, double* __restrict__ part) {
  __shared__ double red[4];
  const int z = blockIdx.y;
  // rows and columns up to 2^17: at most 2^31 runs
  const int64_t cols = G.flip ? G.r : G.k;
  const uint32_t per = (uint32_t)(cols + 7) / 8, n = (uint32_t)(G.flip ? G.k : G.r) * per, step = gridDim.x * 256;
  const T* base = G.p + z * G.stride;
  double sum = 0.0;
  for (uint32_t c0 = blockIdx.x * 256 + threadIdx.x; c0 < n; c0 += 4 * step) {
    Run8<T> r[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t c = c0 + q * step;
      r[q].load(base + (c < n ? c / per * G.ld : 0), c < n ? c % per * 8 : cols, cols);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[8];
      r[q].get(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += (double)v[e] * v[e];
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[(int64_t)z * gridDim.x + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// X and X^T planes from the matrix, scaled by sx / (|G|_F + eps), zeros past its ends: one 64 x 64 tile a workgroup.
// 4096 x 14336 bf16: 117 MB read and 470 MB written in 138 us, 4.3 TB/s, once a call of 11.8 ms.
template <typename T>
__global__ __launch_bounds__(256) void k_orth_load(Dense<const T> G, const double* __restrict__ part, int parts,
                                                   float sx, float eps, int tk, Planes X, Planes Xt) {
  __shared__ float t[64][65];
  const int z = blockIdx.y, i0 = blockIdx.x / tk * 64, k0 = blockIdx.x % tk * 64;
  // the stored tile, rows a0 and columns c0
  const int a0 = G.flip ? k0 : i0, c0 = G.flip ? i0 : k0, rows = G.flip ? G.k : G.r, cols = G.flip ? G.r : G.k;
  Run8<T> r[2];  // under way while the norm is summed
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int w = threadIdx.x + 256 * q, a = w / 8, c = w % 8 * 8;
    const bool in = a0 + a < rows && c0 + c < cols;
    r[q].load(G.p + z * G.stride + (in ? (a0 + a) * G.ld : 0), in ? c0 + c : cols, cols);
  }
  const double f = (double)sx / (__builtin_sqrt(sum_parts(part + (int64_t)z * parts, parts)) + (double)eps);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int w = threadIdx.x + 256 * q, a = w / 8, c = w % 8 * 8;
    float v[8];
    r[q].get(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) t[a][c + e] = (float)((double)v[e] * f);
  }
  __syncthreads();
  const bool flip = G.flip;
  put64(X, z, i0, k0, [&](int i, int k) { return flip ? t[k][i] : t[i][k]; });
  put64(Xt, z, k0, i0, [&](int k, int i) { return flip ? t[k][i] : t[i][k]; });
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

// out = alpha aux + beta a a^T, symmetric: the tiles on and above the diagonal of every matrix of the batch, `per` of
// them a matrix.  The last `rest` of them run as S splits of the K loop each, which write their sums to `part` for
// k_ns_join (they would leave most of a round of workgroups empty).  4096 x 14336: A in 689 us, 1080 TFLOP/s, bound by
// the matrix instructions (busy 61 % at a clock of 1.65 GHz, with 3.2 GB past the L2s; 8192^3 of the library: 1130); 512
// x 1376 fp32: 8 to 11 us, bound by latency.
template <class C>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(2))) void k_ns_sym(
    int tiles, int KT, int full, int rest, int S, Planes a, Planes aux, Planes out, float alpha, float beta,
    float* __restrict__ part) {
  extern __shared__ __align__(16) unsigned char smem[];
  char* lds = reinterpret_cast<char*>(smem);
  const int per = tiles * (tiles + 1) / 2;
  const bool whole = (int)blockIdx.x < full;
  const int u = whole ? xcd_unit(blockIdx.x, full) : xcd_unit(blockIdx.x - full, rest * S);
  const int tile = whole ? u : full + u % rest, sp = whole ? 0 : u / rest, z = tile / per;
  int ti, tj;
  upper_tile(tile % per, tiles, ti, tj);
  const int k0 = whole ? 0 : (int)((int64_t)sp * KT / S), k1 = whole ? KT : (int)((int64_t)(sp + 1) * KT / S);
  Acc<C> acc;
  ns_loop<C>(lds, a.tile(z, ti * C::BM, k0 * C::BK), a.tile(z, tj * C::BN, k0 * C::BK), k1 - k0, ti == tj, acc);
  if (whole) {
    finish_sym<C>(lds, acc, z, ti, tj, aux, out, alpha, beta);
  } else {
    const Planes none{};
    float* o = part + (int64_t)u * C::BM * C::BN;
    ns_store<C>(lds, acc, none, 0.f, 1.f, none, none, 0, [&](const float* st) {
      for (int c = threadIdx.x; c < C::BM * C::BN; c += C::NT) o[c] = st[c / C::BN * C::PITCH + c % C::BN];
    });
  }
}

// alpha aux + beta times the sum over the splits (in order) of a 16 x 64 strip of one of the split BM x BM tiles, and
// its mirror
__global__ __launch_bounds__(256) void k_ns_join(int BM, int tiles, int full, int rest, int S, Planes aux, Planes out,
                                                 float alpha, float beta, const float* __restrict__ part) {
  __shared__ float t[16][65];
  const int per = tiles * (tiles + 1) / 2, cols = BM / 64, strips = BM / 16 * cols, v = blockIdx.x / strips;
  const int si = blockIdx.x % strips / cols * 16, sj = blockIdx.x % cols * 64, z = (full + v) / per;
  int ti, tj;
  upper_tile((full + v) % per, tiles, ti, tj);
  const int c = threadIdx.x % 16 * 4, r = threadIdx.x / 16;
  const int64_t i0 = (int64_t)ti * BM + si, j0 = (int64_t)tj * BM + sj, one = (int64_t)rest * BM * BM;
  const float* P = part + (int64_t)v * BM * BM + (int64_t)(si + r) * BM + sj + c;
  f32x4_v s = {}, x = {};
  int sp = 0;
  for (; sp + 8 <= S; sp += 8) {
    f32x4_v w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = *reinterpret_cast<const f32x4_v*>(P + (sp + e) * one);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += w[e];
  }
  for (; sp < S; ++sp) s += *reinterpret_cast<const f32x4_v*>(P + sp * one);
  if (aux.h) {
    // strips start at multiples of 16 rows, tiles at multiples of 64 columns
    const Planes p = aux.tile(z, i0, j0);
    const int64_t at = r * p.ld + plane_col(c);
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = plane_value(p.h[at + q], p.h[at + kInter + q]);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) t[r][c + q] = alpha * x[q] + beta * s[q];
  __syncthreads();
  // half the threads write the strip in rows, the others its mirror (a column of the strip is a run of 16)
  const bool mirror = threadIdx.x >= 128;
  if (mirror && ti == tj) return;
  const int w = threadIdx.x % 128, row = mirror ? w / 2 : w / 8, col = mirror ? w % 2 * 8 : w % 8 * 8;
  uint32_t y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = pack_hilo(mirror ? t[col + e][row] : t[row][col + e]);
  uint4 h, l;
  split_words(y, 0, h, l);
  // (the mirror's first column, i0, is a multiple of 16: its planes are taken from the 32 below)
  const Planes o = mirror ? out.tile(z, j0, i0 / 32 * 32) : out.tile(z, i0, j0);
  const int64_t at = row * o.ld + plane_col(col + (mirror ? (int)(i0 % 32) : 0));
  put16<true>(o.h + at, h);
  put16<true>(o.h + at + kInter, l);
}

// The tile of unit u of the batch's tm x tn tiles a matrix: matrix, first row, first column.
template <class C> PX_DEV void x_unit(int u, int tm, int tn, int& z, int& m0, int& n0) {
  z = u / (tm * tn);
  int bm, bn;
  x_tile(u % (tm * tn), tm, tn, bm, bn);
  m0 = bm * C::BM;
  n0 = bn * C::BN;
}

// X <- alpha X + beta B X on every tile; X is updated in place (a tile is read by its own workgroup only) and its
// transpose written to the other of two buffers, for the other workgroups still read this one.  4096 x 14336: 1374 us,
// 1050 TFLOP/s, bound by the matrix instructions.
template <class C>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(2))) void k_ns_x(
    int tm, int tn, int KT, Planes B, Planes Xt, Planes X, Planes Xt_out, float alpha, float beta) {
  extern __shared__ __align__(16) unsigned char smem[];
  char* lds = reinterpret_cast<char*>(smem);
  int z, m0, n0;
  x_unit<C>(xcd_unit(blockIdx.x, gridDim.x), tm, tn, z, m0, n0);
  Acc<C> acc;
  ns_loop<C>(lds, B.tile(z, m0, 0), Xt.tile(z, n0, 0), KT, false, acc);
  const Planes o = X.tile(z, m0, n0);
  ns_store<C>(lds, acc, o, alpha, beta, o, Xt_out.tile(z, n0, m0), 0, nullptr);
}

// The last step: alpha X + beta B X to the caller's matrix.
template <class C, typename T>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(2))) void k_ns_out(
    int tm, int tn, int KT, Planes B, Planes Xt, Planes X, Dense<T> O, float alpha, float beta) {
  extern __shared__ __align__(16) unsigned char smem[];
  int z, m0, n0;
  x_unit<C>(xcd_unit(blockIdx.x, gridDim.x), tm, tn, z, m0, n0);
  Acc<C> acc;
  ns_loop<C>(reinterpret_cast<char*>(smem), B.tile(z, m0, 0), Xt.tile(z, n0, 0), KT, false, acc);
  const Planes none{};
  ns_store<C>(reinterpret_cast<char*>(smem), acc, X.tile(z, m0, n0), alpha, beta, none, none, 0,
              [&](const float* st) {
    // lanes run along the stored rows
#pragma unroll 4
    for (int c = threadIdx.x; c < C::BM * C::BN; c += C::NT) {
      const int i = O.flip ? c % C::BM : c / C::BN, j = O.flip ? c / C::BM : c % C::BN;
      const int row = m0 + i, col = n0 + j;
      if (row < O.r && col < O.k) *O.at(z, row, col) = from_f32<T>(st[i * C::PITCH + j]);
    }
  });
}

// workgroups (and 64-bit partial sums) of one matrix's norm: 128 bytes a thread, and no more than fill the GPU
inline int norm_parts(int64_t elems, int es) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(1024, elems * es / (256 * 128)));
}

// allow_lds, once per kernel and GPU: a call makes about 20 launches
template <auto K> hipError_t lds_once(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  e = allow_lds(K, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

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
  // planes of count matrices of rows x cols
  Planes planes(int count, int64_t rows, int64_t cols) {
    Planes p;
    p.ld = 2 * cols;
    p.stride = rows * p.ld;
    p.h = take<f16>((size_t)count * p.stride);
    return p;
  }
};

// The blocks of a step are taken in chunks that bound the workspace, each through all its products.  (Chunks whose
// three buffers would stay in the 256 MB Infinity Cache ran slower, by the rounds of workgroups that they leave
// unfilled: 2.45 ms with 160 MB chunks against 2.10 for 160 blocks of 512 at once.)
constexpr size_t kChunkBytes = size_t(1) << 30;
struct MuonWs {
  int chunk;  // blocks
  double* part;
  BlockInfo* info;
  Planes buf[3];
};
int momentum_parts(int b) { return (int)cdiv((int64_t)b * (b - 1) / 2, kMomentumSlots); }
MuonWs muon_plan(Carve& c, int blocks, int b) {
  MuonWs w{};
  if (b <= 128) return w;
  const int P = (int)round_up(b, 128);
  const int most = (int)std::max<size_t>(1, kChunkBytes / ((size_t)P * P * 12)), chunks = (int)cdiv(blocks, most);
  w.chunk = (int)cdiv(blocks, chunks);
  w.part = c.take<double>((size_t)w.chunk * momentum_parts(b));
  w.info = c.take<BlockInfo>(w.chunk);
  for (Planes& p : w.buf) p = c.planes(w.chunk, P, P);
  return w;
}

// How many of nz blocks of `per` 128 x 128 tiles run on those, the others on 64 x 64 ones: whole rounds of workgroups
// (two a CU), and what is left over of them too where it fills more than 0.6 of a round.  A step in us, the rest on
// 64 x 64 tiles / on 128 x 128: blocks of 512, 0.17 of a round left 770 / 843, 0.46 978 / 1020, 0.73 1759 / 1740, 0.95
// 1312 / 1207; blocks of 256, 0.35 672 / 713, 0.76 838 / 834.  Less than one round runs on 64 x 64 tiles up to 0.75 of
// it: blocks of 256, 0.59 320 / 401, 0.82 417 / 437, 0.94 545 / 466; blocks of 512, 0.23 210 / 355, 0.70 567 / 555,
// 0.78 596 / 580, 0.88 709 / 596.
int muon_wide(int nz, int per) {
  constexpr int slots = 512;
  const int64_t tiles = (int64_t)nz * per, left = tiles % slots;
  if (tiles < slots) return tiles >= 0.75 * slots ? nz : 0;
  return left > 0.6 * slots ? nz : (int)((tiles - left) / per);
}

hipError_t muon_big(MuonTable& t, int b, const MuonK& k, const NsHyper& n, const MuonWs& w, hipStream_t s) {
  constexpr int lds = std::max(NSmall::LDS, NTiny::LDS);
  const int NB = t.first[t.count], n128 = (int)cdiv(b, 128);
  hipError_t e = lds_once<k_ns_skew<false, false>>(lds);
  if (e == hipSuccess) e = lds_once<k_ns_skew<true, false>>(lds);
  if (e == hipSuccess) e = lds_once<k_ns_skew<true, true>>(lds);
  if (e != hipSuccess) return e;
  const float sx = 8.f * pow2_near(std::sqrt((double)b)), ca = (float)n.a, cb = (float)n.b, cc = (float)n.c;
  const unsigned t64 = (unsigned)(2 * n128);
  const int parts = momentum_parts(b);
  for (t.z0 = 0; t.z0 < NB; t.z0 += w.chunk) {
    const int nz = std::min(w.chunk, NB - t.z0);
    k_muon_momentum<<<dim3(parts, nz), 256, 0, s>>>(t, b, k, w.part, w.info);
    k_muon_unpack<<<dim3(t64 * (t64 + 1) / 2, nz), 256, 0, s>>>(t, b, k, w.part, parts, sx, (int)t64, w.buf[0]);
    const int per1 = n128 * (n128 + 1) / 2, per2 = n128 * (2 * n128 + 1), wide = muon_wide(nz, per1);
    const unsigned grid = (unsigned)wide * per1 + (unsigned)(nz - wide) * per2;
    Planes X = w.buf[0], A = w.buf[1];
    const Planes B = w.buf[2], none{};
    for (int it = 0; it < n.steps; ++it) {
      const SkewArgs ga{X, X, none, A, 0.f, kSA / (sx * sx), 0}, gb{A, A, A, B, cb, cc / kSA, 0};
      // X' goes over A, which no product reads any more
      const SkewArgs gx{B, X, X, A, ca, -1.f / kSA, 0x8000u}, gq{B, X, X, none, ca / sx, -1.f / (kSA * sx), 0};
      k_ns_skew<false, false><<<grid, 256, lds, s>>>(ga, w.info, b, n128, wide, k);
      k_ns_skew<true, false><<<grid, 256, lds, s>>>(gb, w.info, b, n128, wide, k);
      if (it + 1 < n.steps)
        k_ns_skew<true, false><<<grid, 256, lds, s>>>(gx, w.info, b, n128, wide, k);
      else
        k_ns_skew<true, true><<<grid, 256, lds, s>>>(gq, w.info, b, n128, wide, k);
      std::swap(X, A);
    }
  }
  return hipGetLastError();
}

template <int P, int W>
hipError_t muon_small(const MuonTable& t, int b, const MuonK& k, const NsHyper& n, hipStream_t s) {
  constexpr int lds = 4 * P * (P + 8) * 2;
  const hipError_t e = lds_once<k_muon_small<P, W>>(lds);
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
  Carve c{reinterpret_cast<char*>(ws)};
  return muon_big(t, b, k, n, muon_plan(c, t.first[count], b), s);
}

namespace {

// How the tiles of one symmetric product run: `full` of them whole, the other `rest` in S splits.
struct SymPlan {
  int tile, tiles;  // tile size, tiles a side
  int full, rest, S;
  size_t part() const { return (size_t)rest * S * tile * tile; }
};
SymPlan sym_plan(int count, int r, int k) {
  SymPlan p{};
  const auto units = [&](int t) { const int64_t n = cdiv(r, t); return count * n * (n + 1) / 2; };
  constexpr int slots = 512;  // two workgroups a CU
  // the whole call in us with tiles of 128 / 64: 36 of 128 (1024 x 4096) 503 / 447; 120 (1920 x 2048) 806 / 707; 136
  // (2048 x 2048) 853 / 829, (2048 x 5461) 1597 / 1597; 210 (2560 x 4096) 1974 / 2065; 528 (4096 x 4096) 4247 / 5219
  p.tile = units(128) >= 200 ? 128 : 64;
  p.tiles = (int)cdiv(r, p.tile);
  const int64_t n = units(p.tile);
  const int KT = (int)cdiv(k, 32), left = (int)(n % slots);
  p.S = 1;
  if (left > 0 && left <= 0.6 * slots) {
    // rounds of workgroups times the K tiles of one, and what the launch that joins them (about 16 K tiles' time) and
    // the partial sums cost
    double best = KT;
    for (int S = 2; S <= 32 && S * 4 <= KT; ++S) {
      const double cost =
          (double)cdiv((int64_t)left * S, slots) * cdiv(KT, S) + 16.0 + 4.0 * S * left / slots + 0.25 * S;
      if (cost < best) {
        best = cost;
        p.S = S;
      }
    }
  }
  p.rest = p.S > 1 ? left : 0;
  p.full = (int)(n - p.rest);
  return p;
}

struct OrthPlan {
  int r, k, rp, kp;
  SymPlan a, b;
  int xtile;  // tile size of X's products
  double* part;
  float* sums;
  Planes X, Xt[2], A, B;
};

OrthPlan orth_plan(Carve& c, int count, int rows, int cols, int dt) {
  OrthPlan p{};
  p.r = std::min(rows, cols);
  p.k = std::max(rows, cols);
  p.a = sym_plan(count, p.r, p.k);
  p.b = sym_plan(count, p.r, p.r);
  const auto units = [&](int t) { return (int64_t)count * cdiv(p.r, t) * cdiv(p.k, t); };
  // the whole call in us with tiles of 128 / 64: 64 of 128 (1024 x 1024) 342 / 261; 144 (1536 x 1536) 506 / 501; 240
  // (1920 x 2048) 689 / 714; 256 (1024 x 4096) 447 / 452; 640 (2560 x 4096) 1970 / 2078; 1024 (4096 x 4096) 4236 /
  // 4940
  // (Tiles of 256 x 256 on 8 waves would need two sets of 128 accumulators a thread, all the registers there are.)
  p.xtile = units(128) >= 200 ? 128 : 64;
  p.rp = (int)round_up(p.r, std::max(p.xtile, p.a.tile));
  p.kp = (int)round_up(p.k, p.xtile);
  p.part = c.take<double>((size_t)count * norm_parts((int64_t)rows * cols, dt == F32 ? 4 : 2));
  p.X = c.planes(count, p.rp, p.kp);
  for (Planes& t : p.Xt) t = c.planes(count, p.kp, p.rp);
  p.A = c.planes(count, p.rp, p.rp);
  p.B = c.planes(count, p.rp, p.rp);
  p.sums = c.take<float>(std::max(p.a.part(), p.b.part()));
  return p;
}

// out = alpha aux + beta a a^T over K columns
template <class C>
hipError_t sym_launch(const SymPlan& p, int K, const Planes& a, const Planes& aux, const Planes& out, float alpha,
                      float beta, float* sums, hipStream_t s) {
  const hipError_t e = lds_once<k_ns_sym<C>>(C::LDS);
  if (e != hipSuccess) return e;
  k_ns_sym<C><<<p.full + p.rest * p.S, C::NT, C::LDS, s>>>(p.tiles, (int)cdiv(K, C::BK), p.full, p.rest, p.S, a, aux,
                                                           out, alpha, beta, sums);
  if (p.rest > 0)
    k_ns_join<<<p.rest * (C::BM / 16) * (C::BM / 64), 256, 0, s>>>(C::BM, p.tiles, p.full, p.rest, p.S, aux, out, alpha,
                                                                 beta, sums);
  return hipGetLastError();
}
hipError_t sym_run(const SymPlan& p, int K, const Planes& a, const Planes& aux, const Planes& out, float alpha,
                   float beta, float* sums, hipStream_t s) {
  if (p.tile == 128) return sym_launch<NSmall>(p, K, a, aux, out, alpha, beta, sums, s);
  return sym_launch<NTiny>(p, K, a, aux, out, alpha, beta, sums, s);
}

// X', or with `last` the caller's matrix
template <class C, typename T>
hipError_t x_launch(const OrthPlan& p, int count, const Planes& cur, const Planes& nxt, bool last, const Dense<T>& O,
                    float alpha, float beta, hipStream_t s) {
  hipError_t e = lds_once<k_ns_x<C>>(C::LDS);
  if (e == hipSuccess) e = lds_once<k_ns_out<C, T>>(C::LDS);
  if (e != hipSuccess) return e;
  const int tm = (int)cdiv(p.r, C::BM), tn = (int)cdiv(p.k, C::BN), KR = (int)cdiv(p.r, C::BK);
  const unsigned grid = (unsigned)(count * tm * tn);
  if (last)
    k_ns_out<C, T><<<grid, C::NT, C::LDS, s>>>(tm, tn, KR, p.B, cur, p.X, O, alpha, beta);
  else
    k_ns_x<C><<<grid, C::NT, C::LDS, s>>>(tm, tn, KR, p.B, cur, p.X, nxt, alpha, beta);
  return hipGetLastError();
}

template <typename T>
hipError_t orth_run(const OrthPlan& p, int count, const Dense<const T>& G, const Dense<T>& O, const NsHyper& n,
                    hipStream_t s) {
  const float sx = 8.f * pow2_near(std::sqrt((double)p.k)), a = (float)n.a, b = (float)n.b, c = (float)n.c;
  const float scale = n.rms > 0 ? (float)(n.rms * std::sqrt((double)p.k)) : 1.f;
  const Planes none{};
  const int parts = norm_parts((int64_t)p.r * p.k, sizeof(T));
  k_orth_norm<T><<<dim3(parts, count), 256, 0, s>>>(G, p.part);
  k_orth_load<T><<<dim3((unsigned)(p.rp / 64) * (p.kp / 64), count), 256, 0, s>>>(G, p.part, parts, sx, (float)n.eps,
                                                                                p.kp / 64, p.X, p.Xt[0]);
  for (int it = 0; it < n.steps; ++it) {
    const Planes &cur = p.Xt[it & 1], &nxt = p.Xt[(it + 1) & 1];
    hipError_t e = sym_run(p.a, p.k, p.X, none, p.A, 0.f, kSA / (sx * sx), p.sums, s);
    if (e == hipSuccess) e = sym_run(p.b, p.r, p.A, p.A, p.B, b, c / kSA, p.sums, s);
    const bool last = it + 1 == n.steps;
    const float al = last ? a * scale / sx : a, be = last ? scale / (kSA * sx) : 1.f / kSA;
    if (e != hipSuccess) return e;
    e = p.xtile == 128 ? x_launch<NSmall, T>(p, count, cur, nxt, last, O, al, be, s)
                       : x_launch<NTiny, T>(p, count, cur, nxt, last, O, al, be, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
hipError_t orth_t(int count, int rows, int cols, int dt, const void* G, int64_t ldg, int64_t sg, void* O, int64_t ldo,
                  int64_t so, const NsHyper& n, void* ws, hipStream_t s) {
  Carve c{reinterpret_cast<char*>(ws)};
  const OrthPlan p = orth_plan(c, count, rows, cols, dt);
  const int flip = rows > cols;
  const Dense<const T> g{reinterpret_cast<const T*>(G), ldg, sg, p.r, p.k, flip};
  const Dense<T> o{reinterpret_cast<T*>(O), ldo, so, p.r, p.k, flip};
  return orth_run<T>(p, count, g, o, n, s);
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
