// Layer norm and RMS norm of token rows, forward and backward.
//
//   S = X (+ R, rounded to the activation dtype);  mu = mean(S) (0 for RMS)
//   rs = 1 / sqrt(mean((S - mu)^2) + eps);  Y = (S - mu) rs w + b
//   xh = (S - mu) rs;  g = dY w
//   dX = rs (g - mean(g) - xh mean(g xh)) (+ dS)   (no mean(g) for RMS)
//   dw = sum_t dY xh;  db = sum_t dY
//
// Both directions are bound by HBM: every activation is read once into
// registers, where the row stays until its outputs are written.  A row belongs
// to TPR threads with E elements each (a wave, or a workgroup whose waves
// exchange their sums through LDS), each thread owning the same columns of
// every row it meets: the weights, and in the backward the column sums dw and
// db, live in its registers over all rows.  The variance is a second sum over
// the registers, around the mean, so that an offset of the row costs no
// digits.  All sums are fp32.
//
// Rows need no alignment beyond their element's: the 16-byte accesses below
// carry their element's alignment, which the memory path of gfx950 serves.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "poetx_internal.h"

namespace {

template <typename T> constexpr int kVecOf = 16 / (int)sizeof(T);

// Elements [c0, c0 + V) of a row of d; zeros past its end.
template <typename T> PX_DEV void load_chunk(const T* __restrict__ row, int c0, int d, T (&v)[kVecOf<T>]) {
  constexpr int V = kVecOf<T>;
  if (c0 + V <= d) {
    __builtin_memcpy(v, row + c0, 16);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = c0 + e < d ? row[c0 + e] : T(0);
  }
}
template <typename T> PX_DEV void store_chunk(T* __restrict__ row, int c0, int d, const T (&v)[kVecOf<T>]) {
  constexpr int V = kVecOf<T>;
  if (c0 + V <= d) {
    __builtin_memcpy(row + c0, v, 16);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c0 + e < d) row[c0 + e] = v[e];
  }
}

// A thread's share of a row: NC chunks of V elements, chunk k at column (k TPR + lane) V.
template <typename T, int TPR, int E> struct Row {
  static constexpr int V = kVecOf<T>, NC = E / V;
  static_assert(E % V == 0, "whole chunks");
  T v[NC][V];
  static PX_DEV int col(int k, int lane) { return (k * TPR + lane) * V; }
  PX_DEV void load(const T* row, int lane, int d) {
#pragma unroll
    for (int k = 0; k < NC; ++k) load_chunk<T>(row, col(k, lane), d, v[k]);
  }
  PX_DEV void store(T* row, int lane, int d) const {
#pragma unroll
    for (int k = 0; k < NC; ++k) store_chunk<T>(row, col(k, lane), d, v[k]);
  }
};

// fp32 parameters of the thread's columns (`none` where the caller has none)
template <typename T, int TPR, int E>
PX_DEV void load_param(const float* p, float none, int lane, int d, float (&w)[E]) {
  using R = Row<T, TPR, E>;
#pragma unroll
  for (int k = 0; k < R::NC; ++k)
#pragma unroll
    for (int e = 0; e < R::V; ++e) {
      const int c = R::col(k, lane) + e;
      w[k * R::V + e] = p && c < d ? p[c] : none;
    }
}

// The sums of N values over the TPR threads of a row, in a fixed order.  Rows
// of more than one wave use `red` (TPR / 64 x N floats a row) and a barrier of
// the workgroup; two calls that follow each other take different buffers, and
// a buffer is used again only after a barrier that every reader of it has
// passed.
template <int TPR, int N> PX_DEV void row_sum(float (&s)[N], float* red) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor(s[i], m);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = (threadIdx.x >> 6) % W;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[wave * N + i] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = red[i];
#pragma unroll
      for (int w = 1; w < W; ++w) t += red[w * N + i];
      s[i] = t;
    }
  }
}

struct FwdArgs {
  const void *X, *R;
  void *S, *Y;
  const float *w, *b;
  float* stats;
  int64_t ldx, ldr, lds, ldy;
  int T, d;
  float eps;
};

// NT threads hold NT / TPR rows at a time; workgroup g takes rows g RPW + sub, + gridDim RPW, ...  Bound by bytes in
// long calls (8192 x 4096 bf16, RMS with a residual: 268 MB in 46.9 us, 5.7 TB/s), by the launch and the two dependent
// sums of a row in short ones (2048 x 512 bf16, layer: 6.9 us; one row of 4096: 4.0 us).
template <typename T, bool RMS, bool RES, int TPR, int E>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_norm_fwd(const FwdArgs a) {
  constexpr int NT = TPR < 256 ? 256 : TPR, RPW = NT / TPR, W = TPR / 64;
  static_assert(TPR == 64 || RPW == 1, "rows of several waves have the workgroup's barriers to themselves");
  using R = Row<T, TPR, E>;
  __shared__ float red[4 * W];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR, d = a.d;
  const T* X = reinterpret_cast<const T*>(a.X);
  const T* Rs = reinterpret_cast<const T*>(a.R);
  T* S = reinterpret_cast<T*>(a.S);
  T* Y = reinterpret_cast<T*>(a.Y);
  const float fd = (float)d;  // the means are quotients, so that a constant row's is exact
  const int step = gridDim.x * RPW;
  int t = blockIdx.x * RPW + sub;
  R x, r;
  // a workgroup's barriers are uniform: TPR > 64 has one row per workgroup
  if (t < a.T) {
    x.load(X + (int64_t)t * a.ldx, lane, d);
    if constexpr (RES) r.load(Rs + (int64_t)t * a.ldr, lane, d);
  }
  float w[E], b[E];
  load_param<T, TPR, E>(a.w, 1.f, lane, d, w);
  if constexpr (!RMS) load_param<T, TPR, E>(a.b, 0.f, lane, d, b);
  for (int par = 0; t < a.T; t += step, par ^= 1) {
    float f[E];
#pragma unroll
    for (int k = 0; k < R::NC; ++k)
#pragma unroll
      for (int e = 0; e < R::V; ++e) {
        if constexpr (RES) x.v[k][e] = from_f32<T>(to_f32<T>(x.v[k][e]) + to_f32<T>(r.v[k][e]));
        f[k * R::V + e] = to_f32<T>(x.v[k][e]);
      }
    if constexpr (RES) {
      x.store(S + (int64_t)t * a.lds, lane, d);
    }
    // the next row's loads fly while this row is summed
    const int nt = t + step;
    if (nt < a.T) {
      x.load(X + (int64_t)nt * a.ldx, lane, d);
      if constexpr (RES) r.load(Rs + (int64_t)nt * a.ldr, lane, d);
    }
    float mean = 0.f;
    if constexpr (!RMS) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < E; ++i) s[0] += f[i];
      row_sum<TPR, 1>(s, red + 2 * par * W);
      mean = s[0] / fd;
#pragma unroll
      for (int k = 0; k < R::NC; ++k)
#pragma unroll
        for (int e = 0; e < R::V; ++e)  // columns past the row's end stay out of the variance
          f[k * R::V + e] = R::col(k, lane) + e < d ? f[k * R::V + e] - mean : 0.f;
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) s[0] += f[i] * f[i];
    row_sum<TPR, 1>(s, red + (2 * par + 1) * W);
    const float rs = 1.f / __builtin_sqrtf(s[0] / fd + a.eps);
    R y;
#pragma unroll
    for (int k = 0; k < R::NC; ++k)
#pragma unroll
      for (int e = 0; e < R::V; ++e) {
        const int i = k * R::V + e;
        float v = f[i] * rs * w[i];
        if constexpr (!RMS) v += b[i];
        y.v[k][e] = from_f32<T>(v);
      }
    y.store(Y + (int64_t)t * a.ldy, lane, d);
    if (lane == 0) {
      if constexpr (RMS) {
        a.stats[t] = rs;
      } else {
        a.stats[t] = mean;
        a.stats[(int64_t)a.T + t] = rs;
      }
    }
  }
}

struct BwdArgs {
  const void *dY, *S, *dS;
  void* dX;
  const float *w, *stats;
  float* part;  // [parts][vecs][d]: the workgroups' column sums
  int64_t ldy, lds, ldds, ldx;
  int T, d;
};

// A workgroup of 1024 threads holds RPW rows at a time: 16 waves keep enough loads in flight for one workgroup a CU,
// and its rows' column sums leave as one row of partial sums (four times the workgroups of a quarter the size, each
// with its partial sums, ran 16384 x 2048 in 65.6 us and 3001 x 1376 in 23.9).  Bound by bytes: 16384 x 2048 bf16 with
// dS, 268 MB in 53.4 us, 5.0 TB/s; 3001 x 1376 bf16, three rows a workgroup, 16.0 us.
constexpr int kBwdThreads = 1024;
template <typename T, bool RMS, bool RES, int TPR, int E>
__global__ __launch_bounds__(kBwdThreads) void k_norm_bwd(const BwdArgs a) {
  constexpr int RPW = kBwdThreads / TPR, W = TPR / 64, VECS = RMS ? 1 : 2;
  using R = Row<T, TPR, E>;
  __shared__ float red[2][RPW][2 * W];
  __shared__ float acc[RPW > 1 ? VECS : 1][RPW > 1 ? TPR * E : 1];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR, d = a.d;
  const T* dY = reinterpret_cast<const T*>(a.dY);
  const T* S = reinterpret_cast<const T*>(a.S);
  const T* dS = reinterpret_cast<const T*>(a.dS);
  T* dX = reinterpret_cast<T*>(a.dX);
  const float* st_rs = RMS ? a.stats : a.stats + a.T;
  const float fd = (float)d;
  float w[E], dw[E], db[RMS ? 1 : E];
  load_param<T, TPR, E>(a.w, 1.f, lane, d, w);
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = 0.f;
  if constexpr (!RMS)
#pragma unroll
    for (int i = 0; i < E; ++i) db[i] = 0.f;
  const int step = gridDim.x * RPW;
  R y, x, r;
  float mean = 0.f, rs = 0.f;
  auto fetch = [&](int u) {
    y.load(dY + (int64_t)u * a.ldy, lane, d);
    x.load(S + (int64_t)u * a.lds, lane, d);
    if constexpr (RES) r.load(dS + (int64_t)u * a.ldds, lane, d);
    if constexpr (!RMS) mean = a.stats[u];
    rs = st_rs[u];
  };
  int t = blockIdx.x * RPW + sub;
  if (t < a.T) fetch(t);
  // every row group of the workgroup takes part in its barriers: the loop runs while the first one has rows
  for (int t0 = blockIdx.x * RPW, par = 0; t0 < a.T; t0 += step, t += step, par ^= 1) {
    const bool live = t < a.T;
    float g[E], xh[E], add[RES ? E : 1];
    const float rst = rs;
    float s[VECS] = {};
    if (live) {
#pragma unroll
      for (int k = 0; k < R::NC; ++k)
#pragma unroll
        for (int e = 0; e < R::V; ++e) {
          const int i = k * R::V + e;
          const float dy = to_f32<T>(y.v[k][e]);
          xh[i] = (to_f32<T>(x.v[k][e]) - mean) * rs;
          if constexpr (RES) add[i] = to_f32<T>(r.v[k][e]);
          g[i] = dy * w[i];
          dw[i] += dy * xh[i];
          if constexpr (!RMS) {
            db[i] += dy;
            s[1] += g[i];
          }
          s[0] += g[i] * xh[i];
        }
    }
    const int nt = t + step;
    if (nt < a.T) fetch(nt);
    row_sum<TPR, VECS>(s, red[par][sub]);
    if (!live) continue;
    const float m0 = s[0] / fd, m1 = RMS ? 0.f : s[VECS - 1] / fd;
    R o;
#pragma unroll
    for (int k = 0; k < R::NC; ++k)
#pragma unroll
      for (int e = 0; e < R::V; ++e) {
        const int i = k * R::V + e;
        float v = rst * (g[i] - m1 - xh[i] * m0);
        if constexpr (RES) v += add[i];
        o.v[k][e] = from_f32<T>(v);
      }
    o.store(dX + (int64_t)t * a.ldx, lane, d);
  }
  // the workgroup's column sums: its rows' partial sums added in the order of `sub`
  if constexpr (RPW > 1) {
    for (int q = 0; q < RPW; ++q) {
      if (sub == q)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int c = i * TPR + lane;  // a place of its own per thread and element
          acc[0][c] = q == 0 ? dw[i] : acc[0][c] + dw[i];
          if constexpr (!RMS) acc[VECS - 1][c] = q == 0 ? db[i] : acc[VECS - 1][c] + db[i];
        }
      __syncthreads();
    }
    if (sub != 0) return;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      dw[i] = acc[0][i * TPR + lane];
      if constexpr (!RMS) db[i] = acc[VECS - 1][i * TPR + lane];
    }
  }
  float* P = a.part + (int64_t)blockIdx.x * VECS * d;
#pragma unroll
  for (int k = 0; k < R::NC; ++k)
#pragma unroll
    for (int e = 0; e < R::V; ++e) {
      const int c = R::col(k, lane) + e;
      if (c < d) {
        P[c] = dw[k * R::V + e];
        if constexpr (!RMS) P[d + c] = db[k * R::V + e];
      }
    }
}

// dw and db: the sums of `parts` rows of n = vecs d columns, 16 columns by 16
// row groups a workgroup, the groups' sums added in order.  Bound by the launch: 256 x 2048 partial sums, 2 MB, 4.6 us.
__global__ __launch_bounds__(256) void k_norm_colsum(const float* __restrict__ part, int parts, int n, int d,
                                                     float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float t[16][17];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  float s = 0.f;
  if (col < n) {
    int p = g;
    for (; p + 7 * 16 < parts; p += 8 * 16) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = part[(int64_t)(p + 16 * k) * n + col];
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
    for (; p < parts; p += 16) s += part[(int64_t)p * n + col];
  }
  t[g][c] = s;
  __syncthreads();
  if (g == 0 && col < n) {
    s = t[0][c];
#pragma unroll
    for (int k = 1; k < 16; ++k) s += t[k][c];
    float* out = col < d ? dw : db;
    if (out) out[col < d ? col : col - d] = s;
  }
}

// The threads and elements per thread of a row of d: 8 elements while 1024 threads hold the row (with 16 a thread,
// half the waves to keep loads in flight, 8192 x 4096 bf16 took 60.3 us forward instead of 54.2).
template <int V> using Int = std::integral_constant<int, V>;
template <bool BWD, typename F> hipError_t by_width(int d, F&& f) {
  if (d <= 64 * 8) return f(Int<64>(), Int<8>());
  if constexpr (BWD)  // rows of two waves share a workgroup (and its barriers) in the backward only
    if (d <= 128 * 8) return f(Int<128>(), Int<8>());
  if (d <= 256 * 8) return f(Int<256>(), Int<8>());
  if (d <= 512 * 8) return f(Int<512>(), Int<8>());
  if (d <= 1024 * 8) return f(Int<1024>(), Int<8>());
  if (d <= 1024 * 16) return f(Int<1024>(), Int<16>());
  return f(Int<1024>(), Int<32>());
}
// rows that a workgroup of the backward holds at a time
int bwd_rows(int d) {
  int n = 1;
  by_width<true>(d, [&](auto tpr, auto) {
    n = kBwdThreads / decltype(tpr)::value;
    return hipSuccess;
  });
  return n;
}

template <typename T, bool RMS, bool RES> hipError_t fwd_t(const FwdArgs& a, hipStream_t s) {
  return by_width<false>(a.d, [&](auto tpr, auto el) {
    constexpr int TPR = decltype(tpr)::value, E = decltype(el)::value, NT = TPR < 256 ? 256 : TPR, RPW = NT / TPR;
    const int64_t groups = ((int64_t)a.T + RPW - 1) / RPW;
    const unsigned grid = (unsigned)std::min<int64_t>(groups, 256 * (2048 / NT));
    k_norm_fwd<T, RMS, RES, TPR, E><<<grid, NT, 0, s>>>(a);
    return hipGetLastError();
  });
}

template <typename T, bool RMS, bool RES> hipError_t bwd_t(const BwdArgs& a, int parts, hipStream_t s) {
  return by_width<true>(a.d, [&](auto tpr, auto el) {
    constexpr int TPR = decltype(tpr)::value, E = decltype(el)::value;
    k_norm_bwd<T, RMS, RES, TPR, E><<<(unsigned)parts, kBwdThreads, 0, s>>>(a);
    return hipGetLastError();
  });
}

template <typename F> hipError_t by_kind(int dt, bool rms, bool res, F&& f) {
  auto k = [&](auto t) {
    if (rms)
      return res ? f(t, std::true_type(), std::true_type()) : f(t, std::true_type(), std::false_type());
    return res ? f(t, std::false_type(), std::true_type()) : f(t, std::false_type(), std::false_type());
  };
  return dt == pxk::BF16 ? k(bf16_t(0)) : k(0.f);
}

}  // namespace

namespace pxk {

int norm_bwd_parts(int64_t T, int d) {
  const int rows = bwd_rows(d);
  return (int)std::min<int64_t>((T + rows - 1) / rows, 256);  // one workgroup a CU
}

hipError_t norm_fwd(int dt, bool rms, int64_t T, int d, float eps, const void* X, int64_t ldx, const void* R,
                    int64_t ldr, const float* w, const float* b, void* S, int64_t lds, void* Y, int64_t ldy,
                    float* stats, hipStream_t s) {
  const FwdArgs a{X, R, S, Y, w, b, stats, ldx, ldr, lds, ldy, (int)T, d, eps};
  return by_kind(dt, rms, R != nullptr, [&](auto t, auto m, auto r) {
    return fwd_t<decltype(t), decltype(m)::value, decltype(r)::value>(a, s);
  });
}

hipError_t norm_bwd(int dt, bool rms, int64_t T, int d, const void* dY, int64_t ldy, const void* S, int64_t lds,
                    const float* w, const float* stats, const void* dS, int64_t ldds, void* dX, int64_t ldx, float* dw,
                    float* db, float* part, hipStream_t s) {
  const int parts = norm_bwd_parts(T, d);
  const BwdArgs a{dY, S, dS, dX, w, stats, part, ldy, lds, ldds, ldx, (int)T, d};
  if (parts > 0) {
    const hipError_t e = by_kind(dt, rms, dS != nullptr, [&](auto t, auto m, auto r) {
      return bwd_t<decltype(t), decltype(m)::value, decltype(r)::value>(a, parts, s);
    });
    if (e != hipSuccess) return e;
  }
  if (!dw && !db) return hipSuccess;
  const int n = (rms ? 1 : 2) * d;
  k_norm_colsum<<<(unsigned)((n + 15) / 16), 256, 0, s>>>(part, parts, n, d, dw, db);
  return hipGetLastError();
}

}  // namespace pxk
