// Rotary positions of token rows (poetx_rope).
//
// A pair (x, y) of a head turns by the angle pos f[j]: 6 fp32 operations for 2 elements read and written once, so the
// kernel is bound by memory.  The angle depends on the token and the pair alone: a workgroup forms the sines and
// cosines of its tokens once, in LDS, and every head of every matrix reads them from there.  Queries and keys of 8192
// tokens with 40 heads of 128 in bf16 (168 MB) take 35.6 us, 4.7 TB/s, the rate of a copy; 28 where the caches hold part.
//
// pos f reaches 2^31 radians, where fp32 has no digit left behind the point.  The angle is formed in turns in fp64,
// whole turns are taken off exactly, and only the rest is rounded to fp32.
#include <algorithm>

#include "common.h"
#include "poetx_internal.h"

namespace {

using namespace pxk;

constexpr int kThreads = 256;

struct RopeArgs {
  RopeSide side[kRopeSides];
  const int32_t* pos;
  const double* freqs;
  int64_t T, first;  // first: the launch's first token
  float amplitude, sign;
  int count, hd, rot, tokens;  // tokens of a workgroup
};

// W elements, from and to any element boundary
template <typename T, int W> PX_DEV void load_w(float (&f)[W], const T* p) {
  T v[W];
  __builtin_memcpy(v, p, sizeof(v));
#pragma unroll
  for (int i = 0; i < W; ++i) f[i] = to_f32<T>(v[i]);
}
template <typename T, int W> PX_DEV void store_w(T* p, const float (&f)[W]) {
  T v[W];
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = from_f32<T>(f[i]);
  __builtin_memcpy(p, v, sizeof(v));
}

// A unit is W pairs, or W of the elements behind rot_dim.  The threads stand as heads x units, so that a thread keeps
// its unit, and the division is done once.
template <typename T, int W, bool PAIRS> __global__ __launch_bounds__(kThreads) void k_rope(RopeArgs a) {
  extern __shared__ float2 turn[];  // [tokens][rot / 2]: cos, sin
  const int half = a.rot / 2;
  const int64_t t0 = a.first + (int64_t)blockIdx.x * a.tokens;
  const int nt = (int)min((int64_t)a.tokens, a.T - t0);
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half;
    const double p = a.pos ? (double)a.pos[t0 + t] : (double)(t0 + t);
    const double turns = p * (a.freqs[i - t * half] * 0.15915494309189533577);  // 1 / (2 pi)
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    turn[i] = make_float2(a.amplitude * c, a.amplitude * a.sign * s);
  }
  __syncthreads();
  const int rot_units = half / W, units = rot_units + (a.hd - a.rot) / W;
  const int lanes = min(units, kThreads);  // threads of one head
  const int h0 = (int)threadIdx.x / lanes, hstep = kThreads / lanes;
  if (h0 >= hstep) return;
  for (int t = 0; t < nt; ++t) {
    const float2* tab = turn + t * half;
    for (int i = 0; i < a.count; ++i) {
      const RopeSide& sd = a.side[i];
      const T* X = static_cast<const T*>(sd.X) + (t0 + t) * sd.ldx;
      T* Y = static_cast<T*>(sd.Y) + (t0 + t) * sd.ldy;
      for (int u = (int)threadIdx.x - h0 * lanes; u < units; u += lanes) {
        if (u >= rot_units) {
          const int c = a.rot + (u - rot_units) * W;
          if (sd.X != sd.Y)
            for (int h = h0; h < sd.heads; h += hstep) {
              T v[W];
              __builtin_memcpy(v, X + h * a.hd + c, sizeof(v));
              __builtin_memcpy(Y + h * a.hd + c, v, sizeof(v));
            }
          continue;
        }
        float2 cs[W];
#pragma unroll
        for (int j = 0; j < W; ++j) cs[j] = tab[u * W + j];
        const int c0 = PAIRS ? 2 * u * W : u * W, c1 = PAIRS ? c0 + W : c0 + half;
        for (int h = h0; h < sd.heads; h += hstep) {
          float p[W], q[W];
          load_w<T, W>(p, X + h * a.hd + c0);
          load_w<T, W>(q, X + h * a.hd + c1);
          float y0[W], y1[W];
#pragma unroll
          for (int j = 0; j < W; ++j) {
            // the elements of pair j in the two runs of W: side by side, or one in each
            const float x = PAIRS ? (2 * j < W ? p[(2 * j) % W] : q[(2 * j) % W]) : p[j];
            const float y = PAIRS ? (2 * j + 1 < W ? p[(2 * j + 1) % W] : q[(2 * j + 1) % W]) : q[j];
            const float rx = x * cs[j].x - y * cs[j].y, ry = y * cs[j].x + x * cs[j].y;
            if (PAIRS) {
              (2 * j < W ? y0 : y1)[(2 * j) % W] = rx;
              (2 * j + 1 < W ? y0 : y1)[(2 * j + 1) % W] = ry;
            } else {
              y0[j] = rx;
              y1[j] = ry;
            }
          }
          store_w<T, W>(Y + h * a.hd + c0, y0);
          store_w<T, W>(Y + h * a.hd + c1, y1);
        }
      }
    }
  }
}

template <typename T, int W> hipError_t launch(RopeArgs a, bool pairs, hipStream_t s) {
  const int64_t most = int64_t(1) << 22;  // workgroups of a launch, whose threads have to stay below 2^32
  const int lds = a.tokens * (a.rot / 2) * (int)sizeof(float2);
  for (a.first = 0; a.first < a.T; a.first += most * a.tokens) {
    const dim3 grid((unsigned)std::min(most, (a.T - a.first + a.tokens - 1) / a.tokens));
    if (pairs)
      k_rope<T, W, true><<<grid, kThreads, lds, s>>>(a);
    else
      k_rope<T, W, false><<<grid, kThreads, lds, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

namespace pxk {

hipError_t rope(int dt, bool pairs, int64_t T, int hd, int rot, const int32_t* pos, const double* freqs,
                float amplitude, bool inverse, int count, const RopeSide* sides, hipStream_t s) {
  if (T == 0) return hipSuccess;
  RopeArgs a;
  for (int i = 0; i < count; ++i) a.side[i] = sides[i];
  a.pos = pos;
  a.freqs = freqs;
  a.T = T;
  a.amplitude = amplitude;
  a.sign = inverse ? -1.f : 1.f;
  a.count = count;
  a.hd = hd;
  a.rot = rot;
  // as many tokens as give every thread an angle, while 1024 workgroups are left
  a.tokens = (int)std::max<int64_t>(1, std::min<int64_t>(kThreads / (rot / 2), T / 1024));
  // 16 bytes an access where the runs are whole numbers of them (65536 tokens of 40 heads of 128: 252 us; by elements 312)
  const int W = dt == BF16 ? 8 : 4;
  const bool wide = (rot / 2) % W == 0 && (hd - rot) % W == 0;
  if (dt == BF16) return wide ? launch<bf16_t, 8>(a, pairs, s) : launch<bf16_t, 1>(a, pairs, s);
  return wide ? launch<float, 4>(a, pairs, s) : launch<float, 1>(a, pairs, s);
}

}  // namespace pxk
