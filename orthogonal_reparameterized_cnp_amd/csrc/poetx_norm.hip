// Layer norm and RMS norm of token rows, forward and backward.
//
//   S = X (+ R, rounded to the activation dtype);  mu = mean(S) (0 for RMS)
//   rs = 1 / sqrt(mean((S - mu)^2) + eps);  Y = (S - mu) rs w + b
//   xh = (S - mu) rs;  g = dY w
//   dX = rs (g - mean(g) - xh mean(g xh)) (+ dS)   (no mean(g) for RMS)
//   dw = sum_t dY xh;  db = sum_t dY
//
// Both directions are bound by HBM: every activation is read once into
// registers, where the row stays until its outputs are written (of the widest
// rows a part spills, see by_width).  A row belongs to TPR threads with E
// elements each (a wave, or a workgroup whose waves
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

typedef uint32_t u32x4_v __attribute__((ext_vector_type(4)));

// The columns of a thread: NC chunks of V, chunk k at min((k TPR + lane) V, d - V).  Only the row's last chunk is moved
// back by the minimum (and those past the row, which hold nothing): its first `skip` columns are its neighbour's,
// loaded and left out.  So loads have no branch of their own for the row's end, and a next row's stay in flight while
// this one is summed.  (With one, every row waited where its paths joined for the loads just issued: backward of 16384
// x 2048 bf16 66 us instead of 52, forward of 1021 x 5461 bf16 21 instead of 13.)
template <typename T, int TPR, int E> struct Cols {
  static constexpr int V = kVecOf<T>, NC = E / V;
  static_assert(E % V == 0, "whole chunks");
  int at[NC], skip[NC], d;
  PX_DEV bool whole() const { return TPR > 64 || d >= V; }  // rows of a chunk at least
  PX_DEV Cols(int lane, int d_) : d(d_) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c0 = (k * TPR + lane) * V;
      at[k] = max(0, min(c0, d - V));
      skip[k] = c0 - at[k];
    }
  }
  PX_DEV bool own(int k, int e) const { return e >= skip[k] && (whole() || e < d); }
};

// A thread's share of a row, as loaded.
template <typename T, int TPR, int E> struct Row {
  using C = Cols<T, TPR, E>;
  static constexpr int V = C::V, NC = C::NC;
  u32x4_v v[NC];
  PX_DEV void load(const T* row, const C& c) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      if (c.whole()) {
        __builtin_memcpy(&v[k], row + c.at[k], 16);
      } else {
        T t[V];
#pragma unroll
        for (int e = 0; e < V; ++e) t[e] = row[min(e, c.d - 1)];
        __builtin_memcpy(&v[k], t, 16);
      }
    }
  }
  PX_DEV void store(T* row, const C& c) const {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      if (c.skip[k] == 0 && c.whole()) {
        __builtin_memcpy(row + c.at[k], &v[k], 16);
      } else if (c.skip[k] < V) {
        T t[V];
        __builtin_memcpy(t, &v[k], 16);
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (c.own(k, e)) row[c.at[k] + e] = t[e];
      }
    }
  }
  PX_DEV void get(int k, float (&f)[V]) const {
    // the compiler would take 16-bit elements apart where they are loaded, and wait for them there
    u32x4_v w = v[k];
    asm volatile("" : "+v"(w));
    T t[V];
    __builtin_memcpy(t, &w, 16);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = to_f32<T>(t[e]);
  }
  PX_DEV void set(int k, const float (&f)[V]) {
    T t[V];
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] = from_f32<T>(f[e]);
    __builtin_memcpy(&v[k], t, 16);
  }
};

// fp32 parameters of the thread's columns (`none` where the caller has none)
template <typename T, int TPR, int E>
PX_DEV void load_param(const float* p, float none, const Cols<T, TPR, E>& c, float (&w)[E]) {
  using C = Cols<T, TPR, E>;
#pragma unroll
  for (int k = 0; k < C::NC; ++k) {
    if (p && c.whole())
      __builtin_memcpy(w + k * C::V, p + c.at[k], C::V * 4);
    else
#pragma unroll
      for (int e = 0; e < C::V; ++e) w[k * C::V + e] = p ? p[min(e, c.d - 1)] : none;
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
// long calls (8192 x 4096 bf16, RMS with a residual: 268 MB from memory in 51.7 us, 5.2 TB/s), by the launch and the
// two dependent sums of a row in short ones (2048 x 512 bf16, layer: 4.1 us; one row of 4096: 2.5 us).
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
  const Cols<T, TPR, E> cols(lane, d);
  R x, r;
  // a workgroup's barriers are uniform: TPR > 64 has one row per workgroup
  if (t < a.T) {
    x.load(X + (int64_t)t * a.ldx, cols);
    if constexpr (RES) r.load(Rs + (int64_t)t * a.ldr, cols);
  }
  float w[E], b[E];
  load_param<T, TPR, E>(a.w, 1.f, cols, w);
  if constexpr (!RMS) load_param<T, TPR, E>(a.b, 0.f, cols, b);
  for (int par = 0; t < a.T; t += step, par ^= 1) {
    float f[E];
#pragma unroll
    for (int k = 0; k < R::NC; ++k) {
      float v[R::V], q[R::V];
      x.get(k, v);
      if constexpr (RES) {
        r.get(k, q);
#pragma unroll
        for (int e = 0; e < R::V; ++e) v[e] += q[e];
        x.set(k, v);
        x.get(k, v);
      }
#pragma unroll
      for (int e = 0; e < R::V; ++e) f[k * R::V + e] = cols.own(k, e) ? v[e] : 0.f;
    }
    if constexpr (RES) x.store(S + (int64_t)t * a.lds, cols);
    // the next row's loads fly while this row is summed
    const int nt = t + step;
    if (nt < a.T) {
      x.load(X + (int64_t)nt * a.ldx, cols);
      if constexpr (RES) r.load(Rs + (int64_t)nt * a.ldr, cols);
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
        for (int e = 0; e < R::V; ++e)  // columns that are not the thread's stay out of the variance
          f[k * R::V + e] = cols.own(k, e) ? f[k * R::V + e] - mean : 0.f;
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) s[0] += f[i] * f[i];
    row_sum<TPR, 1>(s, red + (2 * par + 1) * W);
    const float rs = 1.f / __builtin_sqrtf(s[0] / fd + a.eps);
    R y;
#pragma unroll
    for (int k = 0; k < R::NC; ++k) {
      float v[R::V];
#pragma unroll
      for (int e = 0; e < R::V; ++e) {
        const int i = k * R::V + e;
        v[e] = f[i] * rs * w[i];
        if constexpr (!RMS) v[e] += b[i];
      }
      y.set(k, v);
    }
    y.store(Y + (int64_t)t * a.ldy, cols);
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
// and its rows' column sums leave as one row of partial sums (workgroups of 256 / 512 / 1024, four, two or one a CU,
// whole calls back to back: 16384 x 2048 bf16 with dS 60.8 / 55.1 / 52.9 us, 3001 x 1376 bf16 23.8 / 16.4 / 14.4).
// Bound by bytes: 16384 x 2048, 268 MB at 5.2 TB/s; 3001 x 1376 bf16, three rows a workgroup one after the other, by
// their sums.
constexpr int bwd_threads(int tpr, int e) { return e > 8 ? tpr : 1024 / tpr * tpr; }
template <typename T, bool RMS, bool RES, int TPR, int E>
__global__ __launch_bounds__(bwd_threads(TPR, E)) void k_norm_bwd(const BwdArgs a) {
  constexpr int NT = bwd_threads(TPR, E), RPW = NT / TPR, W = TPR / 64, VECS = RMS ? 1 : 2;
  using R = Row<T, TPR, E>;
  __shared__ float red[2][RPW][2 * W];
  __shared__ float acc[RPW > 1 ? RPW : 1][RPW > 1 ? E : 1][TPR + 8];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR, d = a.d;
  const T* dY = reinterpret_cast<const T*>(a.dY);
  const T* S = reinterpret_cast<const T*>(a.S);
  const T* dS = reinterpret_cast<const T*>(a.dS);
  T* dX = reinterpret_cast<T*>(a.dX);
  const float* st_rs = RMS ? a.stats : a.stats + a.T;
  const float fd = (float)d;
  float w[E], dw[E], db[RMS ? 1 : E];
  const Cols<T, TPR, E> cols(lane, d);
  load_param<T, TPR, E>(a.w, 1.f, cols, w);
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = 0.f;
  if constexpr (!RMS)
#pragma unroll
    for (int i = 0; i < E; ++i) db[i] = 0.f;
  const int step = gridDim.x * RPW;
  R y, x, r;
  float mean = 0.f, rs = 0.f;
  auto fetch = [&](int u) {
    y.load(dY + (int64_t)u * a.ldy, cols);
    x.load(S + (int64_t)u * a.lds, cols);
    if constexpr (RES) r.load(dS + (int64_t)u * a.ldds, cols);
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
      for (int k = 0; k < R::NC; ++k) {
        float vy[R::V], vx[R::V], vr[R::V];
        y.get(k, vy);
        x.get(k, vx);
        if constexpr (RES) r.get(k, vr);
#pragma unroll
        for (int e = 0; e < R::V; ++e) {
          const int i = k * R::V + e;
          const bool own = cols.own(k, e);
          const float dy = own ? vy[e] : 0.f;
          xh[i] = own ? (vx[e] - mean) * rs : 0.f;
          if constexpr (RES) add[i] = vr[e];
          g[i] = dy * w[i];
          dw[i] += dy * xh[i];
          if constexpr (!RMS) {
            db[i] += dy;
            s[1] += g[i];
          }
          s[0] += g[i] * xh[i];
        }
      }
    }
    const int nt = t + step;
    if (nt < a.T) fetch(nt);
    row_sum<TPR, VECS>(s, red[par][sub]);
    if (!live) continue;
    const float m0 = s[0] / fd, m1 = RMS ? 0.f : s[VECS - 1] / fd;
    R o;
#pragma unroll
    for (int k = 0; k < R::NC; ++k) {
      float v[R::V];
#pragma unroll
      for (int e = 0; e < R::V; ++e) {
        const int i = k * R::V + e;
        v[e] = rst * (g[i] - m1 - xh[i] * m0);
        if constexpr (RES) v[e] += add[i];
      }
      o.set(k, v);
    }
    o.store(dX + (int64_t)t * a.ldx, cols);
  }
  float* P = a.part + (int64_t)blockIdx.x * VECS * d;
  if constexpr (RPW > 1) {
    // the workgroup's column sums: its row groups' added in their order, a column a thread (8 words between the rows of
    // `acc` spread a thread's neighbours over the banks; group after group 3001 x 1376 took 1.2 us longer)
    auto join = [&](const float* v, float* out) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < E; ++i) acc[sub][i][lane] = v[i];
      __syncthreads();
      for (int c = threadIdx.x; c < d; c += NT) {
        const int chunk = c / R::V, k = chunk / TPR, e = c - max(0, min(chunk * R::V, d - R::V));
        float t = 0.f;
#pragma unroll
        for (int q = 0; q < RPW; ++q) t += acc[q][k * R::V + e][chunk % TPR];
        out[c] = t;
      }
    };
    join(dw, P);
    if constexpr (!RMS) join(db, P + d);
  } else {
#pragma unroll
    for (int k = 0; k < R::NC; ++k)
#pragma unroll
      for (int e = 0; e < R::V; ++e) {
        const int c = cols.at[k] + e;
        if (cols.own(k, e)) {
          P[c] = dw[k * R::V + e];
          if constexpr (!RMS) P[d + c] = db[k * R::V + e];
        }
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

// The threads and elements per thread of a row of d: 8 elements while 1024 threads hold the row (with 16 and half the
// threads, forward, 8192 x 4096 bf16 with a residual takes 53.2 us instead of 52.0, 8192 x 5461 bf16 63.9 instead of
// 54.2).  768 threads leave two workgroups a CU all the registers they ask for (4096 x 5461 fp32, layer: 44.5 us
// forward instead of 51.8 on 1024, 60 backward instead of 66); the layer norm's forward takes more than 64 registers,
// so that workgroups of 1024 would run one a CU: 16 elements up to 8192 (8192 x 8192 bf16 59 us instead of 80; RMS,
// which fits, fp32 104 instead of 100).  Past 8192 the backward's rows, sums and weights do not fit the 128 registers
// of a workgroup of 1024: 768 threads have 168, 512 have 256 (1000 x 10000 fp32, layer, 1024 / 768 / 512 threads: 111 /
// 45 / 62 us; 2048 x 14336 bf16, RMS with dS, 1024 / 512: 99 / 68).  What still spills on 768 / 512 threads, in
// registers of a thread: layer norm with dS 59 / 191 in fp32 and 6 / 91 in bf16, RMS with dS 12 / 115 and 0 / 13,
// without dS at most 7 / 78 (fp32, layer, with dS: 2048 x 10000 in 132 us, 2.5 TB/s; 2048 x 14336 in 263, 1.8 TB/s).
// Past 16384 the 32 columns of a thread spill in both directions, up to 147 registers in the forward and 181 to 501 in
// the backward (512 x 20000 bf16, layer, backward: 172 us, 0.36 TB/s).
template <int V> using Int = std::integral_constant<int, V>;
template <bool BWD, bool RMS, typename F> hipError_t by_width(int d, F&& f) {
  if (d <= 64 * 8) return f(Int<64>(), Int<8>());
  if constexpr (BWD)  // rows of two waves share a workgroup (and its barriers) in the backward only
    if (d <= 128 * 8) return f(Int<128>(), Int<8>());
  if (d <= 256 * 8) return f(Int<256>(), Int<8>());
  if (d <= 512 * 8) return f(Int<512>(), Int<8>());
  if (d <= 768 * 8) return f(Int<768>(), Int<8>());
  if constexpr (!BWD && !RMS)
    if (d <= 512 * 16) return f(Int<512>(), Int<16>());
  if (d <= 1024 * 8) return f(Int<1024>(), Int<8>());
  if constexpr (BWD) {
    if (d <= 768 * 16) return f(Int<768>(), Int<16>());
    if (d <= 512 * 32) return f(Int<512>(), Int<32>());
  } else {
    if (d <= 1024 * 16) return f(Int<1024>(), Int<16>());
  }
  return f(Int<1024>(), Int<32>());
}
// rows that a workgroup of the backward holds at a time
int bwd_rows(int d) {
  int n = 1;
  by_width<true, false>(d, [&](auto tpr, auto el) {
    constexpr int TPR = decltype(tpr)::value;
    n = bwd_threads(TPR, decltype(el)::value) / TPR;
    return hipSuccess;
  });
  return n;
}

template <typename T, bool RMS, bool RES> hipError_t fwd_t(const FwdArgs& a, hipStream_t s) {
  return by_width<false, RMS>(a.d, [&](auto tpr, auto el) {
    constexpr int TPR = decltype(tpr)::value, E = decltype(el)::value, NT = TPR < 256 ? 256 : TPR, RPW = NT / TPR;
    const int64_t groups = ((int64_t)a.T + RPW - 1) / RPW;
    const unsigned grid = (unsigned)std::min<int64_t>(groups, 256 * (2048 / NT));
    k_norm_fwd<T, RMS, RES, TPR, E><<<grid, NT, 0, s>>>(a);
    return hipGetLastError();
  });
}

template <typename T, bool RMS, bool RES> hipError_t bwd_t(const BwdArgs& a, int parts, hipStream_t s) {
  return by_width<true, RMS>(a.d, [&](auto tpr, auto el) {
    constexpr int TPR = decltype(tpr)::value, E = decltype(el)::value;
    k_norm_bwd<T, RMS, RES, TPR, E><<<(unsigned)parts, bwd_threads(TPR, E), 0, s>>>(a);
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
