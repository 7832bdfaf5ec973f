// Log probabilities of given tokens, entropy and top alternatives of rows of logits, and the gradient of the logits
// (poetx_logp_fwd, poetx_logp_bwd).
//
// Forward: one pass over the row.  With c = scale log2(e), every thread keeps the running maximum m of its logits, the
// sum s of 2^y and the sum w of y 2^y, y = c (x - m); a new maximum takes both over:
//     d = c (m - m'):  w' = 2^d (w + d s),  s' = 2^d s.
// Then lse = scale m + ln 2 log2 s, and the entropy is ln 2 (log2 s - w / s): logits are only subtracted from logits,
// which is exact near the maximum, and the sums do not overflow where a mask holds the type's lowest value (lse may,
// with a scale above 1, and is held within the range).  The row is read once and nothing is written but a few words, so
// memory bounds the kernel while there are rows for the whole card: 4096 rows of 32000 logits in bf16 (262 MB) 47 to 55
// us, 4.8 to 5.5 TB/s; 2.1 GB at 5.5, which is this card's rate of reading.  With fewer, a row is cut into parts whose
// sums a second launch joins: one row of 131072 with 8 alternatives takes 7.7 + 6.7 us.
//
// The top alternatives come from the same pass.  A logit and its index make one 64-bit key, larger for larger logits
// and for lower indexes among equal ones; lane i of a wave keeps the wave's i-th largest key so far.  A key that beats
// the last of them is put in by one ballot (its place) and one shift; of n keys in any order about top (1 + ln(n /
// top)) do, so nearly all of them cost one comparison (those that do follow each other: 8 alternatives of the 4096 rows
// 106 us).  The first keys would all do: they are held against the top-th largest of the lanes' maxima first (23.5 ->
// 15.6 us for that row).
#include <algorithm>

#include "common.h"
#include "poetx_internal.h"

namespace {

using namespace pxk;

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kMost = 3.402823466e38f;  // the largest fp32

struct Sums {
  float m, s, w;
};
PX_DEV float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
PX_DEV float finite_or_0(float m) { return m == -INFINITY ? 0.f : m; }
// c (m - to), held above where 2^ of it is 0 anyway, so that its products with the sums stay finite
PX_DEV float distance(float m, float to, float c) { return fmaxf((m - to) * c, -1e4f); }
PX_DEV Sums join(const Sums& a, const Sums& b, float c) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  const float at = finite_or_0(r.m), da = distance(a.m, at, c), db = distance(b.m, at, c);
  const float ea = exp2_of(da), eb = exp2_of(db);
  r.s = a.s * ea + b.s * eb;
  r.w = ea * (a.w + da * a.s) + eb * (b.w + db * b.s);
  return r;
}
PX_DEV Sums shuffled(const Sums& a, int x) { return Sums{__shfl_xor(a.m, x), __shfl_xor(a.s, x), __shfl_xor(a.w, x)}; }

// a 32-bit value in the order of the logits: -0 as 0, NaN above all
PX_DEV uint32_t order(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  if (x != x) return 0xffffffffu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
PX_DEV float unorder(uint32_t k) {
  return k == 0xffffffffu ? NAN : __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
PX_DEV uint64_t key_of(float x, int i) { return ((uint64_t)order(x) << 32) | (uint32_t)~i; }
PX_DEV int index_of(uint64_t k) { return (int)~(uint32_t)k; }

PX_DEV uint64_t lane_value(uint64_t v, int lane) {
  return ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32) |
         (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// v of the lane below (lane 0: any value): one instruction a word, where a shuffle goes through LDS
PX_DEV uint64_t from_lane_below(uint64_t v) {
  constexpr int kWaveShr1 = 0x138;
  const int lo = __builtin_amdgcn_update_dpp(0, (int)v, kWaveShr1, 0xf, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), kWaveShr1, 0xf, 0xf, false);
  return ((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo;
}
// The n-th largest of the lanes' values, bit by bit.
PX_DEV uint32_t nth_largest(uint32_t v, int n) {
  uint64_t in = ~0ull;  // the lanes that agree with the result in the bits so far
  uint32_t r = 0;
#pragma unroll
  for (int b = 31; b >= 0; --b) {
    const uint64_t ones = __ballot(v >> b & 1) & in;
    const int k = __popcll(ones);
    const bool one = k >= n;
    in = one ? ones : in & ~ones;
    n -= one ? 0 : k;
    r |= (uint32_t)one << b;
  }
  return r;
}

// The wave's `top` largest keys, lane i the i-th; 0 (below every key) where there is none.
struct TopList {
  uint64_t mine = 0, last = 0;  // this lane's; the smallest that is kept
  int top;
  PX_DEV explicit TopList(int n) : top(n) {}
  // k is the same in every lane and above `last`
  PX_DEV void put(uint64_t k) {
    const int at = __popcll(__ballot(mine > k));
    const uint64_t up = from_lane_below(mine);
    const int lane = threadIdx.x & 63;
    mine = lane < at ? mine : lane == at ? k : up;
    last = lane_value(mine, top - 1);
  }
  // every lane's k, the lanes one after another; keys under `floor` are known to be too small
  PX_DEV void offer(uint64_t k, uint64_t floor = 0) {
    if (k < floor) k = 0;
    uint64_t better = __ballot(k > last);
    while (better) {
      put(lane_value(k, __builtin_ctzll(better)));
      better = __ballot(k > last) & ~((2ull << __builtin_ctzll(better)) - 1);
    }
  }
  // a list in memory, from the largest down
  PX_DEV void offer_list(const uint64_t* l) {
    const int lane = threadIdx.x & 63;
    const uint64_t k = lane < top ? l[lane] : 0;
    for (int i = 0; i < top; ++i) {
      const uint64_t x = lane_value(k, i);
      if (x <= last) break;
      put(x);
    }
  }
};

struct LogpOut {
  const int32_t* target;
  float *logp, *lse, *entropy;
  int32_t* ids;
  float* lps;
};
// the same from row r on
LogpOut rows_from(const LogpOut& o, int64_t r, int top) {
  const auto at = [](auto* p, int64_t n) { return p ? p + n : p; };
  return LogpOut{at(o.target, r), at(o.logp, r), at(o.lse, r), at(o.entropy, r), at(o.ids, r * top), at(o.lps, r * top)};
}

// what one row's sums and list say; wave 0 of the workgroup calls it
template <typename T>
PX_DEV void finish(const Sums& v, const TopList& best, const T* x, int64_t row, int V, int top, float scale,
                   const LogpOut& o) {
  const int lane = threadIdx.x & 63;
  // no finite logit: s = 0 and the log is -infinity
  const float ls = log2f(v.s);
  const float m = finite_or_0(v.m), log_sum = kLn2 * ls;
  if (lane == 0) {
    // A scale above 1 takes finite logits out of the range.  Their lse stays at its end: infinities are those of rows
    // without a finite logit, and the backward tells them apart by that.
    const float l = m * scale + log_sum;
    o.lse[row] = v.s > 0.f ? fminf(fmaxf(l, -kMost), kMost) : l;
    if (o.entropy) o.entropy[row] = v.s == 0.f ? 0.f : kLn2 * (ls - v.w / v.s);
    if (o.logp) {
      const int t = o.target[row];
      float lp = 0.f;
      if (t >= 0 && t < V) lp = v.s == 0.f ? -INFINITY : (to_f32<T>(x[t]) - m) * scale - log_sum;
      o.logp[row] = lp;
    }
  }
  if (lane < top) {
    o.ids[row * top + lane] = index_of(best.mine);
    const float l = unorder((uint32_t)(best.mine >> 32));
    o.lps[row * top + lane] = l == -INFINITY ? -INFINITY : (l - m) * scale - log_sum;
  }
}

// Part blockIdx.x % parts of row blockIdx.x / parts: columns [part, part + 1) * span.  With several parts, its sums and
// list go to `part_sums` and `part_keys`.
template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void k_logp_fwd(const T* X, int64_t ldx, int V, int top, float scale, int parts,
                                                       int span, float4* part_sums, uint64_t* part_keys, LogpOut o) {
  constexpr int W = 16 / (int)sizeof(T), UNROLL = 4;
  const int64_t row = blockIdx.x / parts;
  const int part = blockIdx.x % parts;
  const T* x = X + row * ldx;
  const int c0 = part * span, c1 = min(V, c0 + span);
  const float c = scale * kLog2e;
  Sums v{-INFINITY, 0.f, 0.f};
  TopList best(TOP ? top : 1);
  const auto take = [&](const float (&f)[W], int at) {
    float m = v.m;
#pragma unroll
    for (int i = 0; i < W; ++i) m = fmaxf(m, f[i]);
    const float base = finite_or_0(m), d = distance(v.m, base, c), e = exp2_of(d);
    v.w = e * (v.w + d * v.s);
    v.s = e * v.s;
    v.m = m;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float y = (f[i] - base) * c, p = exp2_of(y);
      v.s += p;
      v.w += fmaxf(y, -3e38f) * p;  // y = -infinity has p = 0
    }
    if (TOP) {
      // the last that is kept, or -infinity; an equal logit may have a lower index
      const float bar = best.last ? unorder((uint32_t)(best.last >> 32)) : -INFINITY;
      bool any = false;
#pragma unroll
      for (int i = 0; i < W; ++i) any |= !(f[i] < bar);
      if (__ballot(any)) {
        // While the list is not full: of the lanes' largest logits here the top-th, below which no logit can be among
        // the `top` largest.  It spares most of the insertions that an empty list would take.
        uint64_t floor = 0;
        if (best.last == 0) {
          uint32_t most = 0;
#pragma unroll
          for (int i = 0; i < W; ++i) most = max(most, at + i < c1 ? order(f[i]) : 0u);
          floor = (uint64_t)nth_largest(most, top) << 32;
        }
#pragma unroll
        for (int i = 0; i < W; ++i) best.offer(at + i < c1 ? key_of(f[i], at + i) : 0, floor);
      }
    }
  };
  const auto load = [&](float (&f)[W], int at) {
    if (at + W <= c1) {
      T t[W];
      __builtin_memcpy(t, x + at, sizeof(t));
#pragma unroll
      for (int i = 0; i < W; ++i) f[i] = to_f32<T>(t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) f[i] = at + i < c1 ? to_f32<T>(x[at + i]) : -INFINITY;
    }
  };
  // the same trips for every lane of a wave, which the list's ballots need
  int at = c0;
  for (; at + UNROLL * kThreads * W <= c1; at += UNROLL * kThreads * W) {
    float f[UNROLL][W];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) load(f[u], at + (u * kThreads + (int)threadIdx.x) * W);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) take(f[u], at + (u * kThreads + (int)threadIdx.x) * W);
  }
  for (; at < c1; at += kThreads * W) {
    float f[W];
    load(f, at + (int)threadIdx.x * W);
    take(f, at + (int)threadIdx.x * W);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = join(v, shuffled(v, d), c);
  __shared__ Sums sums[kWaves];
  __shared__ uint64_t keys[kWaves][kLogpTop];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (lane == 0) sums[wave] = v;
  if (TOP && lane < top) keys[wave][lane] = best.mine;
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int i = 1; i < kWaves; ++i) {
    v = join(v, sums[i], c);
    if (TOP) best.offer_list(keys[i]);
  }
  if (parts == 1) {
    finish<T>(v, best, x, row, V, TOP ? top : 0, scale, o);
    return;
  }
  if (lane == 0) part_sums[blockIdx.x] = make_float4(v.m, v.s, v.w, 0.f);
  if (TOP && lane < top) part_keys[(int64_t)blockIdx.x * top + lane] = best.mine;
}

// joins the parts of row blockIdx.x, their sums in one order
template <typename T>
__global__ __launch_bounds__(kThreads) void k_logp_join(const T* X, int64_t ldx, int V, int top, float scale,
                                                        int parts, const float4* part_sums, const uint64_t* part_keys,
                                                        LogpOut o) {
  const int64_t row = blockIdx.x;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  TopList best(top ? top : 1);
  // all parts' keys, 64 at a time; the first ones' top-th is a floor for the rest
  const uint64_t* list = part_keys + row * parts * top;
  for (int x = wave * 64; x < parts * top; x += kThreads) {
    const uint64_t k = x + lane < parts * top ? list[x + lane] : 0;
    const uint64_t floor = best.last ? 0 : (uint64_t)nth_largest((uint32_t)(k >> 32), top) << 32;
    best.offer(k, floor);
  }
  __shared__ uint64_t keys[kWaves][kLogpTop];
  if (lane < top) keys[wave][lane] = best.mine;
  __syncthreads();
  if (wave > 0) return;
  const float c = scale * kLog2e;
  Sums v{-INFINITY, 0.f, 0.f};
  for (int p = lane; p < parts; p += 64) {
    const float4 f = part_sums[row * parts + p];
    v = join(v, Sums{f.x, f.y, f.z}, c);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = join(v, shuffled(v, d), c);
  if (top)
    for (int i = 1; i < kWaves; ++i) best.offer_list(keys[i]);
  finish<T>(v, best, X + row * ldx, row, V, top, scale, o);
}

// dX of columns [part, part + 1) * span of a row: every element read and written once, so memory bounds it (524 MB in bf16
// 107 us, 4.9 TB/s; 408 MB in fp32 88 us, 4.6; a copy on this card 4.7)
template <typename T, bool ENT>
__global__ __launch_bounds__(kThreads) void k_logp_bwd(const T* X, int64_t ldx, int V, float scale, int parts, int span,
                                                       const int32_t* target, const float* lse, const float* entropy,
                                                       const float* dlogp, const float* dentropy, T* dX, int64_t lddx) {
  constexpr int W = 16 / (int)sizeof(T), UNROLL = 2;
  const int64_t row = blockIdx.x / parts;
  const int part = blockIdx.x % parts;
  const T* x = X + row * ldx;
  T* dx = dX + row * lddx;
  const int c0 = part * span, c1 = min(V, c0 + span);
  // the row's values on the way together, none behind a test of another
  const float l = lse[row], H = ENT ? entropy[row] : 0.f, dh = ENT ? dentropy[row] : 0.f, dl = target ? dlogp[row] : 0.f;
  int t = target ? target[row] : -1;
  if (t < 0 || t >= V) t = -1;
  const float a = t >= 0 && l != -INFINITY ? scale * dl : 0.f, b = ENT && l != -INFINITY ? scale * dh : 0.f;
  // no finite logit, or nothing asked for: the gradient is 0 whatever the row holds (NaN in a batch's padding)
  const bool none = a == 0.f && b == 0.f;
  const float h = none ? 0.f : H;
  // log p of logits beyond the range in a row whose lse is held at its end; others keep what the fma gives
  const float most = l == kMost ? 0.f : INFINITY;
  const auto grad = [&](float f, int at) {
    float y = none ? -INFINITY : f * scale - l;
    y = y > most ? most : y;  // NaN stays
    const float p = exp2_of(y * kLog2e);
    float g = -a * p;
    if (ENT) g -= b * (p * (fmaxf(y, -3e38f) + h));
    return at == t ? g + a : g;
  };
  const auto load = [&](T (&v)[W], int at) {
    if (at + W <= c1) __builtin_memcpy(v, x + at, sizeof(v));
    else
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (at + i < c1) v[i] = x[at + i];
  };
  const auto put = [&](T (&v)[W], int at) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = from_f32<T>(grad(to_f32<T>(v[i]), at + i));
    if (at + W <= c1) __builtin_memcpy(dx + at, v, sizeof(v));
    else
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (at + i < c1) dx[at + i] = v[i];
  };
  for (int at = c0 + (int)threadIdx.x * W; at < c1; at += UNROLL * kThreads * W) {
    T v[UNROLL][W] = {};
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) load(v[u], at + u * kThreads * W);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) put(v[u], at + u * kThreads * W);
  }
}

// Parts of a row: enough for four workgroups a CU while a part keeps `least` columns; `span` is a multiple of 1024.  131072
// logits with 8 alternatives: one row 15.8 us in parts, 45 in one; 64 rows 25 and 51; the gradient of 8 rows 7.3 and 9.3.
struct Cut {
  int parts, span;
};
Cut cut(int64_t T, int V, int least) {
  const int64_t want = std::min<int64_t>((1024 + T - 1) / T, (V + least - 1) / least);
  const int span = (int)round_up((V + want - 1) / want, 1024);
  return Cut{(V + span - 1) / span, span};
}
constexpr int kFwdLeast = 2048, kBwdLeast = 4096;
constexpr int64_t kRowsAtOnce = 1 << 22;  // rows of a launch, whose threads have to stay below 2^32

}  // namespace

namespace pxk {

size_t logp_ws_bytes(int dt, int64_t T, int V, int top) {
  (void)dt;
  if (T == 0) return 0;
  const Cut k = cut(T, V, kFwdLeast);
  return k.parts == 1 ? 0 : (size_t)T * k.parts * (16 + 8 * (size_t)top);
}

template <typename T>
static hipError_t fwd(int64_t rows, int V, int top, float scale, const void* Xv, int64_t ldx, const LogpOut& o,
                      void* ws, hipStream_t s) {
  const T* X = static_cast<const T*>(Xv);
  const Cut k = cut(rows, V, kFwdLeast);
  float4* sums = static_cast<float4*>(ws);
  uint64_t* keys = reinterpret_cast<uint64_t*>(sums + rows * k.parts);
  for (int64_t r = 0; r < rows; r += kRowsAtOnce) {  // one launch where there are parts
    const dim3 grid((unsigned)(std::min(rows - r, kRowsAtOnce) * k.parts));
    const T* x = X + r * ldx;
    const LogpOut to = rows_from(o, r, top);
    if (top)
      k_logp_fwd<T, true><<<grid, kThreads, 0, s>>>(x, ldx, V, top, scale, k.parts, k.span, sums, keys, to);
    else
      k_logp_fwd<T, false><<<grid, kThreads, 0, s>>>(x, ldx, V, 0, scale, k.parts, k.span, sums, keys, to);
  }
  if (k.parts > 1)
    k_logp_join<T><<<dim3((unsigned)rows), kThreads, 0, s>>>(X, ldx, V, top, scale, k.parts, sums, keys, o);
  return hipGetLastError();
}

hipError_t logp_fwd(int dt, int64_t T, int V, int top, float scale, const void* X, int64_t ldx, const int32_t* target,
                    float* logp, float* lse, float* entropy, int32_t* top_ids, float* top_logp, void* ws,
                    hipStream_t s) {
  if (T == 0) return hipSuccess;
  const LogpOut o{target, logp, lse, entropy, top_ids, top_logp};
  return dt == BF16 ? fwd<bf16_t>(T, V, top, scale, X, ldx, o, ws, s) : fwd<float>(T, V, top, scale, X, ldx, o, ws, s);
}

template <typename T>
static hipError_t bwd(int64_t rows, int V, float scale, const void* X, int64_t ldx, const int32_t* target,
                      const float* lse, const float* entropy, const float* dlogp, const float* dentropy, void* dX,
                      int64_t lddx, hipStream_t s) {
  const Cut k = cut(rows, V, kBwdLeast);
  const auto at = [](auto* p, int64_t r) { return p ? p + r : p; };
  for (int64_t r = 0; r < rows; r += kRowsAtOnce) {
    const dim3 grid((unsigned)(std::min(rows - r, kRowsAtOnce) * k.parts));
    const T* x = static_cast<const T*>(X) + r * ldx;
    T* dx = static_cast<T*>(dX) + r * lddx;
    if (dentropy)
      k_logp_bwd<T, true><<<grid, kThreads, 0, s>>>(x, ldx, V, scale, k.parts, k.span, at(target, r), lse + r,
                                                    at(entropy, r), at(dlogp, r), at(dentropy, r), dx, lddx);
    else
      k_logp_bwd<T, false><<<grid, kThreads, 0, s>>>(x, ldx, V, scale, k.parts, k.span, at(target, r), lse + r,
                                                     at(entropy, r), at(dlogp, r), at(dentropy, r), dx, lddx);
  }
  return hipGetLastError();
}

hipError_t logp_bwd(int dt, int64_t T, int V, float scale, const void* X, int64_t ldx, const int32_t* target,
                    const float* lse, const float* entropy, const float* dlogp, const float* dentropy, void* dX,
                    int64_t lddx, hipStream_t s) {
  if (T == 0) return hipSuccess;
  return dt == BF16 ? bwd<bf16_t>(T, V, scale, X, ldx, target, lse, entropy, dlogp, dentropy, dX, lddx, s)
                    : bwd<float>(T, V, scale, X, ldx, target, lse, entropy, dlogp, dentropy, dX, lddx, s);
}

}  // namespace pxk
