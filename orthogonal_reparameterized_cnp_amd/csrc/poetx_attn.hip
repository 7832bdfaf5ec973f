// Attention of packed sequences and its backward (poetx_attn_fwd, poetx_attn_bwd).
//
// Every product runs on the 32 x 32 MFMA instructions, oriented so that a lane owns one query (forward, dQ) or one key
// (dK, dV) in all of them.  An accumulator of these instructions holds, in lane l, column l % 32 at the rows
//     row(e) = 8 (e / 4) + 4 (l / 32) + e % 4,   e < 16,
// and the second operand of the next product wants 8 values of the summed index per lane, column l % 32.  A sum does
// not mind the order of its terms: elements 8 c .. 8 c + 7 of the accumulator are used as they stand, and the first
// operand's fragment is read for the same rows (16 c + 4 (l / 32) + {0 .. 3, 8 .. 11}).  So probabilities and score
// gradients go from one product to the next without leaving their lane:
//     forward   S^T = K Q^T       O^T += V^T P^T
//     dQ        S^T = K Q^T,  dP^T = V dO^T       dQ^T += K^T G^T
//     dK, dV    S = Q K^T,    dP = dO V^T         dV^T += dO^T P,  dK^T += Q^T G
// and the softmax's maximum, sum and rescaling are a lane's own, with one exchange between the wave's halves.
//
// bf16 takes v_mfma_f32_32x32x16_bf16; fp32 takes eight v_mfma_f32_32x32x2_f32 for the same 16 terms, on the same
// fragments, so that both types share the kernels.
//
// Scores, softmax, sums and accumulators are fp32.  bf16 rounds P and the score gradients once each, as operands: the
// matrix instructions take no other, and a rounding of 2^-9 of each term is what rounding the result costs as well (the
// results of 2 x 4096 causal tokens are 1.7e-3 off in the norm in O, 2.3e-3 in the gradients; rounding alone: 1.66e-3).
//
// Figures below are of one MI355X at 2 x 4096 causal tokens, 32 query heads over 8 of 128 columns, bf16, where they name
// nothing else.
#include <algorithm>

#include "kernel_util.h"

namespace {

using namespace pxk;

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr unsigned kAtOnce = 512;  // workgroups that the card holds of the bf16 forward and dQ, two a CU (of dK, dV one)
constexpr int kRows = 32 * kWaves;  // rows of a workgroup: queries (forward, dQ) or keys (dK, dV), 32 a wave

PX_DEV float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
// a wave's number, known to be the same in all its lanes
PX_DEV int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
// f of the values of lanes l and l ^ 32
template <class F> PX_DEV float both_halves(float x, const F& f) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
PX_DEV float sum_halves(float x) { return both_halves(x, [](float a, float b) { return a + b; }); }
PX_DEV float max_halves(float x) { return both_halves(x, [](float a, float b) { return fmaxf(a, b); }); }

// ---- types -----------------------------------------------------------------
typedef float f32x8_v __attribute__((ext_vector_type(8)));
typedef short v4i16_t __attribute__((ext_vector_type(4)));
template <typename T> struct FragOf;
template <> struct FragOf<bf16_t> { typedef bf16x8_v type; };
template <> struct FragOf<float> { typedef f32x8_v type; };
template <typename T> using Frag = typename FragOf<T>::type;

PX_DEV void mma(f32x16_v& acc, const bf16x8_v& a, const bf16x8_v& b) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0);
}
PX_DEV void mma(f32x16_v& acc, const f32x8_v& a, const f32x8_v& b) {
#pragma unroll
  for (int e = 0; e < 8; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], acc, 0, 0, 0);
}

// elements 8 c .. 8 c + 7 of an accumulator as an operand
template <typename T> PX_DEV Frag<T> to_frag(const f32x16_v& v, int c);
template <> PX_DEV bf16x8_v to_frag<bf16_t>(const f32x16_v& v, int c) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = f2bf2(v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
  bf16x8_v f;
  __builtin_memcpy(&f, w, 16);
  return f;
}
template <> PX_DEV f32x8_v to_frag<float>(const f32x16_v& v, int c) {
  f32x8_v f;
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = v[8 * c + i];
  return f;
}

// what the rounding of elements 8 c .. 8 c + 7 to `f` left
template <typename T> PX_DEV Frag<T> rest_of(const f32x16_v& v, int c, const Frag<T>& f) {
  f32x16_v r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = v[8 * c + i] - (float)f[i];
  return to_frag<T>(r, 0);
}

// row of accumulator element e, in the half of lanes that begins with row 0 (the other's is 4 higher)
constexpr int acc_row(int e) { return 8 * (e / 4) + e % 4; }

// ---- tiles of token rows in LDS --------------------------------------------
// bf16: [rows][D] in 16-byte chunks, chunk c of row r at c ^ swz(r).  The two low bits of the row choose among the
// 64-byte groups of a row (four of them for D = 128, two and the row's parity for D = 64), so that both the 16-byte
// reads of 16 rows and the transposing reads of 4 rows x 64 bytes touch every bank once.
// fp32: [rows][D + 4] (reads of 32 bytes from 16 rows touch every bank equally).
//
// A lane reads at offsets that it keeps in two registers (Lane) and that every fragment changes by constants: bits of the
// chunk by exclusive or, rows of 16 and tiles by an immediate.
struct Lane {
  int along, across;
  PX_DEV Lane operator+(int bytes) const { return Lane{along + bytes, across + bytes}; }  // bytes: a multiple of 256
  // the same to the compiler as if it changed here: the fragments' offsets are formed where they are used (an operation
  // each) instead of being held in a register each over the whole loop
  PX_DEV Lane here() const {
    Lane l = *this;
    asm volatile("" : "+v"(l.along), "+v"(l.across));
    return l;
  }
};
template <typename T, int D> struct Rows;
template <int D> struct Rows<bf16_t, D> {
  static constexpr int CPR = D / 8;
  static PX_DEV int swz(int r) {
    return D == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  }
  static constexpr int bytes(int rows) { return rows * D * 2; }
  static PX_DEV void put(char* t, int r, int c, const bf16_t (&v)[8]) {
    __builtin_memcpy(t + 16 * (r * CPR + (c ^ swz(r))), v, 16);
  }
  static PX_DEV Lane lane_at() {
    const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31, s = lane & 15;
    const int row = 4 * h + (s >> 2), chunk = 2 * ((lane >> 4) & 1) + ((s & 3) >> 1);
    return Lane{2 * D * r + 16 * (h ^ swz(r)), 2 * D * row + 16 * (chunk ^ swz(row)) + 8 * (s & 1)};
  }
  // columns 16 kk + 8 (lane / 32) .. + 7 of row r0 + lane % 32
  static PX_DEV bf16x8_v along(const char* t, const Lane& l, int r0, int kk) {
    return *reinterpret_cast<const bf16x8_v*>(t + (l.along ^ (32 * kk)) + 2 * D * r0);
  }
  // column c0 + lane % 32 of rows r0 + 4 (lane / 32) + {0 .. 3, 8 .. 11}
  static PX_DEV bf16x8_v across(const char* t, const Lane& l, int r0, int c0) {
    v4i16_t p[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const char* a = t + (l.across ^ (2 * c0) ^ (32 * q)) + 2 * D * (r0 + 8 * q);
      p[q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16_t*)(a));
    }
    bf16x8_v f;
    __builtin_memcpy(&f, p, 16);
    return f;
  }
};
template <int D> struct Rows<float, D> {
  static constexpr int P = D + 4;
  static constexpr int bytes(int rows) { return rows * P * 4; }
  static PX_DEV void put(char* t, int r, int c, const float (&v)[8]) {
    float* p = reinterpret_cast<float*>(t) + r * P + 8 * c;
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
  static PX_DEV Lane lane_at() {
    const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
    return Lane{4 * (r * P + 8 * h), 4 * (4 * h * P + r)};
  }
  static PX_DEV f32x8_v along(const char* t, const Lane& l, int r0, int kk) {
    const float4* p = reinterpret_cast<const float4*>(t + l.along + 4 * (r0 * P + 16 * kk));
    const float4 a = p[0], b = p[1];
    return f32x8_v{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  }
  static PX_DEV f32x8_v across(const char* t, const Lane& l, int r0, int c0) {
    const float* p = reinterpret_cast<const float*>(t + l.across + 4 * (r0 * P + c0));
    f32x8_v f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = p[(i + (i & 4)) * P];
    return f;
  }
};

// Kernels are built for C columns, the head's rounded up.  bf16 has C = 32, 64, 96 and 128 and multiplies with as many,
// in tiles whose rows hold 64 or 128 for the sake of the banks; fp32, whose products take longer than to ask for each
// whether the head reaches it, has 64 and 128.
template <typename T, int C> using RowsOf = Rows<T, sizeof(T) == 4 ? C : C <= 64 ? 64 : 128>;

// whether the columns from c on are multiplied with
template <typename T> PX_DEV bool within(int c, int hd) { return sizeof(T) == 2 || c < hd; }

// How tiles come to LDS: through registers (any type, head and alignment), by direct copies, which take rows of heads of a
// multiple of 8 columns (96 columns: forward 1300 us through registers, 250 by copies), and by direct copies of heads that fill the
// rows, which need not ask where the head ends (16 tokens over 20k keys: 39.2 us with the question, 36.3 without).
enum How { kStaged, kDirect, kWhole };

// 8 elements from column c of a head's row, zeros behind its end and for absent rows
template <int HOW, typename T> PX_DEV void load8(T (&v)[8], const T* row, bool there, int c, int hd) {
  if (there && c + 8 <= hd) {
    __builtin_memcpy(v, row + c, sizeof(v));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = HOW != kWhole && there && c + i < hd ? row[c + i] : T(0);
  }
}
// rows [r0, r0 + N) of a sequence's `n`, into an LDS tile by way of registers: any type, head and alignment
template <typename T, int C, int N, int THREADS = kThreads> struct Staged {
  static constexpr int K = C / 8, ALL = N * K, EACH = (ALL + THREADS - 1) / THREADS;
  static PX_DEV bool in(int x) { return ALL % THREADS == 0 || x < ALL; }
  T v[EACH][8];
  PX_DEV void load(const T* base, int64_t ld, int r0, int n, int hd) {
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int x = i * THREADS + (int)threadIdx.x, r = x / K, c = x % K;
      load8<kStaged>(v[i], base + (int64_t)(r0 + r) * ld, in(x) && r0 + r < n, 8 * c, hd);
    }
  }
  PX_DEV void put(char* tile) const {
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int x = i * THREADS + (int)threadIdx.x;
      if (in(x)) RowsOf<T, C>::put(tile, x / K, x % K, v[i]);
    }
  }
};
// The same by direct global -> LDS copies, 16 bytes a lane, for bf16 heads of a multiple of 8 columns in rows aligned to
// 16 bytes (pitches of up to kDmaLd).  Rows behind the last repeat it; what is computed from them is masked.  Columns
// behind the head are left alone: zero_tail() clears them once.
constexpr int64_t kDmaLd = 1 << 23;  // a tile's rows lie within 32 bits
// `BYTES` from base + at of each lane to the LDS address t + BYTES * lane.  The compiler holds the builtin for a write to any
// LDS that the transposing reads may read, and waits in front of those for all copies in flight.  Where that is too early,
// OWN is assembly, of which it counts nothing: copies_done() or a wait of the kernel's own has to stand before the reads.
// The assembly changes m0, which the compiler holds for its own and lets no clobber name: a kernel takes all its copies in
// one of the two ways, and has nothing else that needs m0.
template <int BYTES, bool OWN> PX_DEV void copy_to_lds(char* t, const char* base, uint32_t at) {
  const auto lds = (__attribute__((address_space(3))) char*)t;
  if constexpr (!OWN && BYTES == 16)
    __builtin_amdgcn_global_load_lds(base + at, (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
  else if constexpr (!OWN)
    __builtin_amdgcn_global_load_lds(base + at, (__attribute__((address_space(3))) void*)lds, 4, 0, 0);
  else if constexpr (BYTES == 16)  // with the wait states between writes of the scalar registers and this use of them
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"((uint32_t)(uintptr_t)lds), "v"(at),
                 "s"(base) : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, %2" ::"s"((uint32_t)(uintptr_t)lds), "v"(at),
                 "s"(base) : "memory");
}
// This wave's copies.  Not even the builtin's are waited for at a barrier, and a wave that has nothing to compute with a
// tile would come to the next barrier without having waited anywhere.
PX_DEV void copies_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
template <int C, int N, int W, bool OWN> struct DmaRows {
  typedef RowsOf<bf16_t, C> R;
  static constexpr int K = R::CPR, RPW = 64 / K, STEP = W * RPW;  // rows of a wave's copy, of the W waves'
  int r, lane;  // this lane's row in the first copy
  PX_DEV explicit DmaRows(int wave) : r(wave * RPW + ((int)threadIdx.x & 63) / K), lane((int)threadIdx.x & 63) {}
  // rows [r0, r0 + N) of the `n` at base; `wave` as above
  PX_DEV void copy(char* tile, const bf16_t* base, int64_t ld, int r0, int n, int hd, int wave) const {
    static_assert(N % STEP == 0, "whole copies");
    char* t = tile + wave * 1024;
    const char* g = reinterpret_cast<const char*>(base + r0 * ld);
    const int pitch = 2 * (int)ld, last = n - 1 - r0;
#pragma unroll
    for (int i = 0; i < N / STEP; ++i) {
      const int row = r + i * STEP, c = 16 * (lane % K ^ R::swz(row));
      if (hd < 8 * K && c >= 2 * hd) continue;
      if (last >= N - 1)
        put(t + i * W * 1024, g + (int64_t)i * STEP * pitch, (uint32_t)(r * pitch + c));
      else
        put(t + i * W * 1024, g, (uint32_t)(min(row, last) * pitch + c));
    }
  }
  static PX_DEV void put(char* t, const char* base, uint32_t at) { copy_to_lds<16, OWN>(t, base, at); }
};
// the columns behind the head, of `rows` rows of an LDS tile, by `threads` threads of which this is the x-th
template <int C> PX_DEV void zero_tail(char* tile, int rows, int hd, int x, int threads) {
  const int k = (C - hd) / 8;  // chunks of 8
  const bf16_t zeros[8] = {};
  for (int i = x; i < rows * k; i += threads) RowsOf<bf16_t, C>::put(tile, i / k, hd / 8 + i % k, zeros);
}
// the operand fragments of one row, held in registers
template <typename T, int C, int HOW>
PX_DEV void row_frags(Frag<T> (&f)[C / 16], const T* row, bool there, int hd, int lane) {
#pragma unroll
  for (int kk = 0; kk < C / 16; ++kk) {
    T v[8];
    load8<HOW>(v, row, there, 16 * kk + 8 * (lane >> 5), hd);
    __builtin_memcpy(&f[kk], v, sizeof(v));
  }
}
// The fragments are there: the compiler, which does not count the copies to LDS, waits for all loads in flight where it
// first needs them, and that has to be before the loop.
template <typename T, int N> PX_DEV void settle(Frag<T> (&f)[N]) {
#pragma unroll
  for (int kk = 0; kk < N; ++kk) asm volatile("" : "+v"(f[kk]));
}
// a lane's accumulator column as row elements: 4 consecutive of them at a time
template <typename T, int C, int HOW>
PX_DEV void store_row(T* row, const f32x16_v (&acc)[C / 32], float scale, int hd, int lane) {
#pragma unroll
  for (int d = 0; d < C / 32; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int c = 32 * d + 8 * g + 4 * (lane >> 5);
      T v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = from_f32<T>(acc[d][4 * g + i] * scale);
      if (c + 4 <= hd) {
        __builtin_memcpy(row + c, v, sizeof(v));
      } else if constexpr (HOW != kWhole) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < hd) row[c + i] = v[i];
      }
    }
}

// ---- sequences -------------------------------------------------------------
struct Side {
  const int32_t* cu;
  int64_t rows, each;  // each: rows of a sequence where cu is null
};
struct AttnArgs {
  const void *Q, *K, *V, *O, *dO;
  int64_t ldq, ldk, ldv, ldo, lddo;
  void *out, *out2;  // O; dQ; dK and dV
  int64_t ldout, ldout2;
  float *lse, *rows;  // rows: the backward's lse and D of every query, [2][heads][Tq]; the parts of few rows, pairs of
                      // maximum and sum and from part_head on their O
  float* parts;       // the shares' dK and dV, [shares][2][kv_heads][Tk][C]
  Side q, k;
  int batch, heads, group, window;
  int hd, row_hd;  // columns of a head; row_hd: in the rows that are copied straight to LDS, hd or its multiple of 8 above
  int part;    // keys of a workgroup in the forward of few rows
  int shares;  // workgroups that share the query heads of a key head in dK and dV
  bool causal;
  float scale;
  int64_t slots, part_head;
  int64_t join0;  // the first query and head of a launch that joins
};
// first row of sequence s (s = batch: behind the last), held within the rows whatever the offsets say
PX_DEV int64_t first_row(const Side& x, int s) {
  if (!x.cu) return x.each * s;
  return min(max((int64_t)x.cu[s], (int64_t)0), x.rows);
}
struct Seq {
  int64_t q0, k0;
  int nq, nk;
};
PX_DEV Seq sequence(const AttnArgs& a, int s) {
  Seq r;
  r.q0 = first_row(a.q, s);
  r.k0 = first_row(a.k, s);
  r.nq = (int)max(first_row(a.q, s + 1) - r.q0, (int64_t)0);
  r.nk = (int)max(first_row(a.k, s + 1) - r.k0, (int64_t)0);
  return r;
}
// The last sequence s that f(s) holds for, or the first; f holds up to some sequence.  64 candidates at a time.
template <class F> PX_DEV int last_seq(int batch, const F& f) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = batch;  // it is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 63) / 64;
    const bool at = lane * step < n && f(lo + lane * step);
    const int k = max((int)__popcll(__ballot(at)) - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}
PX_DEV int seq_of_row(const Side& x, int batch, int64_t row) {
  return last_seq(batch, [&](int s) { return first_row(x, s) <= row; });
}
// The sequence and the tile of `slot`: sequence s of rows [a, b) has the slots from a / R + s on, and the ones up to
// b / R + s are enough for its ceil((b - a) / R) tiles.  So the host needs no length, and a workgroup no prefix sum.
PX_DEV int find_seq(const Side& x, int batch, int64_t slot, int R, int* tile) {
  const auto begin = [&](int s) { return (int64_t)((uint32_t)first_row(x, s) / (uint32_t)R) + s; };
  const int s = last_seq(batch, [&](int s) { return begin(s) <= slot; });
  *tile = (int)(slot - begin(s));
  return s;
}

// The head of workgroup p of a tile's: the query heads of a key head are kv_heads apart, so that with the 8 or 16 key heads
// of usual models they run on one XCD, whose L2 they read the keys from (forward 290 us, with the heads in order 297).
PX_DEV int head_of(const AttnArgs& a, int p) {
  const int kv_heads = a.heads / a.group;
  return p % kv_heads * a.group + p / kv_heads;
}

// The keys [lo, hi) that the query at `place` sees.
struct Sees {
  int lo, hi;
  // the same relative to this lane's row 0 of a tile that begins at j, to compare constants with
  PX_DEV Sees from(int j) const {
    const int at = j + 4 * (((int)threadIdx.x >> 5) & 1);
    return Sees{lo - at, hi - at};
  }
  PX_DEV bool has(int x) const { return x >= lo && x < hi; }
  // bit x: has(x), x < 32
  PX_DEV uint32_t bits() const {
    const auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };
    return below(hi) & ~below(lo);
  }
};
PX_DEV Sees keys_of(const AttnArgs& a, int place, int nk) {
  Sees r;
  r.lo = a.window ? max(place - a.window + 1, 0) : 0;
  r.hi = a.causal ? min(place + 1, nk) : a.window ? (int)min((int64_t)place + a.window, (int64_t)nk) : nk;
  return r;
}
// The places [lo, hi) of the queries that see key j, within [p0, p1).
PX_DEV Sees places_of(const AttnArgs& a, int j, int p0, int p1) {
  Sees r;
  r.lo = a.causal ? max(j, p0) : a.window ? max(j - a.window + 1, p0) : p0;
  r.hi = a.window ? (int)min((int64_t)j + a.window, (int64_t)p1) : p1;
  return r;
}

// What the 32 rows of a wave see together: some of them, and each of them.
struct Span {
  Sees some, each;
  PX_DEV bool any(int lo, int hi) const { return lo < some.hi && hi > some.lo; }
  PX_DEV bool all(int lo, int hi) const { return lo >= each.lo && hi <= each.hi; }
};
// Keys of the queries first .. end, of which there are some.
PX_DEV Span keys_of_rows(const AttnArgs& a, int first, int end, const Seq& sq) {
  const Sees f = keys_of(a, first + sq.nk - sq.nq, sq.nk), e = keys_of(a, end + sq.nk - sq.nq, sq.nk);
  return Span{{f.lo, e.hi}, {e.lo, f.hi}};
}
// Keys of the queries first .. first + 31 of a wave; no key for all of them where some do not exist.
PX_DEV Span keys_of_wave(const AttnArgs& a, int first, const Seq& sq) {
  if (first >= sq.nq) return Span{{0, 0}, {0, 0}};
  Span w = keys_of_rows(a, first, min(first + 31, sq.nq - 1), sq);
  if (first + 31 >= sq.nq) w.each = Sees{0, 0};
  return w;
}

// The n-th tile of R rows in the order in which the workgroups start, which is that of falling work in causal sequences:
// the k-th tile of a sequence (`ends`: counted from its first row; else from its last) attends to about k tiles, and the
// tiles of equal k stand side by side.  So the short ones fill the card's end, however the lengths are mixed.  Of up to
// 64 sequences the order is exact: with f(k) tiles of the k-th class and above, a lane a class,
//     f(k) = sum over the sequences of max(tiles - k, 0);
// more sequences are taken as equal ones, and so are those of a launch that the card takes at once (`order` false), which
// has nothing to fill (the 60M layer's forward 9.0 us, in order 9.4).  16 sequences of 7 to 2048 tokens, 16 heads: forward
// 170 -> 151 us, backward 540 -> 522 against equal ones.  Returns the sequence, with *tile < 0 where there is none.
PX_DEV int tile_of(const Side& x, int batch, int64_t slots, int64_t n, int R, bool order, bool ends, int* tile) {
  if (!order || batch > 64) {
    const int64_t per = slots / batch, t = n / batch;
    if (t < per) n = n % batch * per + t;
    return find_seq(x, batch, ends ? slots - 1 - n : n, R, tile);
  }
  const int lane = threadIdx.x & 63;
  const int rows = lane < batch ? (int)max(first_row(x, lane + 1) - first_row(x, lane), (int64_t)0) : 0;
  const int tiles = (rows + R - 1) / R;
  int most = 0;
  for (int s = 0; s < batch; ++s) most = max(most, __builtin_amdgcn_readlane(tiles, s));
  const auto f = [&](int k) {
    int sum = 0;
    for (int s = 0; s < batch; ++s) sum += max(__builtin_amdgcn_readlane(tiles, s) - k, 0);
    return sum;
  };
  int k = 0;  // the class: the last with f(k) > n
  for (int step = (most + 63) / 64; step > 0; step = step > 1 ? (step + 63) / 64 : 0) {
    const uint64_t in = __ballot(f(k + lane * step) > n);
    *tile = -1;
    if (!in) return 0;
    k += (__popcll(in) - 1) * step;
  }
  if (most == 0) {
    *tile = -1;
    return 0;
  }
  const int nth = (int)n - f(k + 1);
  const uint64_t in = __ballot(tiles > k);
  const int s = __builtin_ctzll(__ballot(tiles > k && __popcll(in & ((1ull << lane) - 1)) == nth));
  *tile = ends ? k : __builtin_amdgcn_readlane(tiles, s) - 1 - k;
  return s;
}

// f(offset of the K tile, which the V tile follows, first key) over the tiles of the keys [j0, j1), which are the same for
// the whole workgroup.
template <typename T, int C, int HOW, int KT, int THREADS = kThreads, class F>
PX_DEV void over_tiles(char* lds, const T* K, int64_t ldk, const T* V, int64_t ldv, int n, int hd, int j0, int j1,
                       const F& f) {
  typedef RowsOf<T, C> R;
  const auto at = [&](int x) { return lds + x * R::bytes(KT); };
  if constexpr (HOW != kStaged) {
    if (j0 >= j1) return;
    const int wave = wave_id();
    const DmaRows<C, KT, kWaves, false> dma(wave);
    const auto copy = [&](int x, int j) __attribute__((always_inline)) {
      dma.copy(at(x), K, ldk, j, n, hd, wave);
      dma.copy(at(x + 1), V, ldv, j, n, hd, wave);
    };
    copy(0, j0);
    zero_tail<C>(lds, 4 * KT, hd, (int)threadIdx.x, kThreads);
    for (int j = j0, x = 0; j < j1; j += KT, x ^= 2) {
      copies_done();
      __syncthreads();  // this tile is there, and the other buffer is done with
      if (j + KT < j1) copy(2 - x, j + KT);
      f(x * R::bytes(KT), j);
    }
  } else if constexpr (KT <= 64) {
    // the next tile's rows come into registers while this one is computed with
    Staged<T, C, KT, THREADS> k, v;
    const auto load = [&](int j) __attribute__((always_inline)) {
      k.load(K, ldk, j, n, hd);
      v.load(V, ldv, j, n, hd);
    };
    if (j0 < j1) load(j0);
    for (int j = j0; j < j1; j += KT) {
      __syncthreads();
      k.put(at(0));
      v.put(at(1));
      __syncthreads();
      if (j + KT < j1) load(j + KT);
      f(0, j);
    }
  } else {  // too many rows for that
    for (int j = j0; j < j1; j += KT) {
      __syncthreads();
      for (int x = 0; x < KT; x += 32) {
        Staged<T, C, 32> k, v;
        k.load(K, ldk, j + x, n, hd);
        v.load(V, ldv, j + x, n, hd);
        k.put(at(0) + R::bytes(x));
        v.put(at(1) + R::bytes(x));
      }
      __syncthreads();
      f(0, j);
    }
  }
}

// ---- forward ---------------------------------------------------------------
template <typename T> constexpr int kTile = sizeof(T) == 2 ? 64 : 32;  // keys (queries for dK, dV) of an LDS tile

// Softmax of one wave's queries over the tiles so far: maximum m (of the raw scores), sum l of this half's keys.  The
// maximum is only taken over where it has grown by more than kSlack (in units of log2 p): until then p may reach
// 2^kSlack, which costs no digits, and the accumulators need no rescaling (forward 291 us; rescaled at every tile, 306).
constexpr float kSlack = 8.f;

// O of 128 queries of one head, 32 a wave: 64 accumulator registers and 32 of q leave room for two waves a SIMD, whose
// products and exponentials then stand against each other; with 32 keys a tile and three waves it is 317 us.  The next
// tile's copies run during this one's work.  285 us, 960 TFLOP/s; 2 x 4096 without a mask 550 us, 1000 TFLOP/s: the
// matrix pipe is busy 52% of the time and the vector pipe nearly as long (counters; no bank conflicts).  The two of a
// tile follow each other within a wave, and two waves hide it in part.

// fp32 has a second group of four waves, which takes the other half of each tile's keys: a wave's products are eight times
// bf16's, and with one group a SIMD had one wave of them and nobody to work while it staged the next tile and took its
// softmax (32 heads of 128: 2048 tokens 338 -> 314 us, 2 x 4096 2562 -> 2350; 64 columns 228 -> 171; six sequences of up to
// 1000 with 9 heads of 75 columns, fewer workgroups than CUs, 72 -> 61).
template <typename T> constexpr int kFwdGroups = sizeof(T) == 2 ? 1 : 2;
template <typename T, int C, int HOW>
__global__ __launch_bounds__(kThreads * kFwdGroups<T>, HOW ? 2 : 1) void k_attn_fwd(AttnArgs a) {
  constexpr int G = kFwdGroups<T>, PART = kTile<T>, KT = PART * G, NB = PART / 32, BUFS = HOW ? 2 : 1;
  typedef RowsOf<T, C> R;
  __shared__ __align__(16) char lds[BUFS * 2 * R::bytes(KT)];
  const int lane = threadIdx.x & 63, wave = wave_id() % kWaves, group = wave_id() / kWaves, hd = HOW == kWhole ? C : a.hd;
  const int head = head_of(a, blockIdx.x % a.heads);
  int tile;
  const Seq sq =
      sequence(a, tile_of(a.q, a.batch, a.slots, blockIdx.x / a.heads, kRows, gridDim.x > kAtOnce, true, &tile));
  const int w0 = tile * kRows;
  if (tile < 0 || w0 >= sq.nq) return;
  const int shift = sq.nk - sq.nq, i = w0 + 32 * wave + (lane & 31);  // this lane's query
  const bool live = i < sq.nq;
  const int row_hd = HOW == kWhole ? C : a.row_hd;
  const T* K = static_cast<const T*>(a.K) + sq.k0 * a.ldk + (int64_t)(head / a.group) * row_hd;
  const T* V = static_cast<const T*>(a.V) + sq.k0 * a.ldv + (int64_t)(head / a.group) * row_hd;
  Frag<T> q[C / 16];
  row_frags<T, C, HOW>(q, static_cast<const T*>(a.Q) + (sq.q0 + i) * a.ldq + (int64_t)head * hd, live, hd, lane);
  const Sees see = live ? keys_of(a, i + shift, sq.nk) : Sees{0, 0};
  const int last = min(w0 + kRows, sq.nq) - 1;
  const int j0 = keys_of(a, w0 + shift, sq.nk).lo / KT * KT, j1 = keys_of(a, last + shift, sq.nk).hi;
  const Span w = keys_of_wave(a, w0 + 32 * wave, sq);
  const float c = a.scale * kLog2e;
  const Lane lane_at = R::lane_at();
  f32x16_v acc[C / 32] = {};
  float m = -INFINITY, l = 0.f;
  const auto step = [&](int tile, int j, auto masked) __attribute__((always_inline)) {
    const Lane at = (lane_at + tile).here();
    const char *const tk = lds, *const tv = lds + R::bytes(KT);
    f32x16_v s[NB] = {};
#pragma unroll
    for (int kk = 0; kk < C / 16; ++kk)
      if (within<T>(16 * kk, hd))
#pragma unroll
        for (int b = 0; b < NB; ++b) mma(s[b], R::along(tk, at, 32 * b, kk), q[kk]);
    float top = -INFINITY;
    const Sees on = see.from(j);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if constexpr (decltype(masked)::value) s[b][e] = on.has(32 * b + acc_row(e)) ? s[b][e] : -INFINITY;
        top = fmaxf(top, s[b][e]);
      }
    top = max_halves(top);
    if (__any((top - m) * c > kSlack)) {  // a first key: top - m is infinite
      const float was = m;
      m = fmaxf(m, top);
      const float keep = exp2_of((was - (m == -INFINITY ? 0.f : m)) * c);
      l *= keep;
#pragma unroll
      for (int d = 0; d < C / 32; ++d) acc[d] *= keep;
    }
    const float base = m == -INFINITY ? 0.f : m;  // no key so far
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        // fp32 keeps the exact difference; bf16's p has fewer digits than one fma leaves
        s[b][e] = sizeof(T) == 4 ? exp2_of((s[b][e] - base) * c) : exp2_of(fmaf(s[b][e], c, -base * c));
        l += s[b][e];
      }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Frag<T> p = to_frag<T>(s[b], h);
#pragma unroll
        for (int d = 0; d < C / 32; ++d)
          if (within<T>(32 * d, hd)) mma(acc[d], R::across(tv, at, 32 * b + 16 * h, 32 * d), p);
      }
  };
  over_tiles<T, C, HOW, KT, kThreads * G>(lds, K, a.ldk, V, a.ldv, sq.nk, row_hd, j0, j1,
                                          [&](int tile, int j) __attribute__((always_inline)) {
                                            j += PART * group, tile += R::bytes(PART) * group;
                                            if (w.all(j, j + PART)) step(tile, j, std::false_type());
                                            else if (w.any(j, j + PART)) step(tile, j, std::true_type());
                                          });
  if constexpr (G == 2) {  // the first group's waves take the second's maxima, sums and O
    static_assert(kWaves * 64 * (C / 2 + 2) * 4 <= sizeof(lds), "the exchange fits");
    float* x = reinterpret_cast<float*>(lds) + wave * 64 * (C / 2 + 2) + lane;
    __syncthreads();
    if (group == 1) {
#pragma unroll
      for (int d = 0; d < C / 32; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[(16 * d + e) * 64] = acc[d][e];
      x[(C / 2) * 64] = m;
      x[(C / 2 + 1) * 64] = l;
    }
    __syncthreads();
    if (group == 1) return;
    const float was = m, other = x[(C / 2) * 64];
    m = fmaxf(m, other);
    const float base = m == -INFINITY ? 0.f : m, keep = exp2_of((was - base) * c), more = exp2_of((other - base) * c);
    l = l * keep + x[(C / 2 + 1) * 64] * more;
#pragma unroll
    for (int d = 0; d < C / 32; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[d][e] = acc[d][e] * keep + x[(16 * d + e) * 64] * more;
  }
  if (!live) return;
  l = sum_halves(l);
  store_row<T, C, HOW>(static_cast<T*>(a.out) + (sq.q0 + i) * a.ldout + (int64_t)head * hd, acc, l == 0.f ? 0.f : 1.f / l,
                  hd, lane);
  if (lane < 32) a.lse[(int64_t)head * a.q.rows + sq.q0 + i] = l == 0.f ? -INFINITY : m * a.scale + kLn2 * log2f(l);
}

// ---- forward of few rows ---------------------------------------------------
// With one or a few queries per sequence the keys are read for little work, and there are too few tiles of 128 queries for
// the card.  Here a tile is 32 rows, a row one query of one of the query heads that share a key head (so that its keys are
// read once for all of them), and the four waves take 32 keys each of a tile of 128.  By direct copies a wave has its own
// piece of LDS and waits for nobody: what bounds the kernel is how many bytes are under way, and waves that load and
// compute at different times keep more of them there than workgroups in step.  (Heads of 128 columns take 264 to 296
// registers in bf16 and 323 in fp32, so that one workgroup stands on a CU; up to 96 columns, in fp32 64, it is two or
// three.)  A wave's next keys are copied
// as soon as these are multiplied, during the softmax, and its next values during the next product (64 tokens over 2048
// keys each 145 -> 130 us).  A workgroup stands for `part` keys of a sequence.  It leaves the maximum, the sum and the
// unscaled O that they give the sequence's rows, and k_attn_join adds the parts in their order.  Where a sequence has more
// rows than a tile all the same, its workgroups share the tiles instead, each with all keys.
//
// HBM bounds it, from some 100 MB of keys on: 64 tokens over 8192 keys each (8 key heads of 128, 2.1 GB) 430 us, 5.0 TB/s,
// what reading alone reaches; 16 over 1 to 8192 (112 MB) 33.5 us with the join (5), one over 100000 91 us, where the start
// and end of a launch and parts of unequal sequences count.  fp32, which stages the keys through registers: 16 over 4096
// each (537 MB) 183 us, 2.9 TB/s, and one over 100000 (819 MB) 259.
constexpr int kFewRows = 32, kFewKeys = 32 * kWaves;
template <typename T, int C> struct Few {
  static constexpr int TILES = 2 * RowsOf<T, C>::bytes(kFewKeys);
  static constexpr int JOIN = kWaves * 64 * (C / 2 + 2) * 4;
  static constexpr int LDS = TILES > JOIN ? TILES : JOIN;
};
PX_DEV int parts_of(const AttnArgs& a, const Seq& sq) { return max((sq.nk + a.part - 1) / a.part, 1); }
// where the O of part slot and key head `kv` is among the parts, in rows of C floats; its maxima and sums lie before
// them all, as pairs
PX_DEV int64_t part_row(const AttnArgs& a, int64_t slot, int kv) {
  return (slot * (a.heads / a.group) + kv) * kFewRows;
}
template <typename T, int C, int HOW> __global__ __launch_bounds__(kThreads) void k_attn_few(AttnArgs a) {
  constexpr int KT = kFewKeys;
  typedef RowsOf<T, C> R;
  extern __shared__ __align__(16) char lds[];
  const int lane = threadIdx.x & 63, wave = wave_id(), hd = HOW == kWhole ? C : a.hd, kv_heads = a.heads / a.group;
  const int kv = (int)(blockIdx.x % kv_heads);
  const int64_t slot = blockIdx.x / kv_heads;
  int part;
  const Seq sq = sequence(a, find_seq(a.k, a.batch, slot, a.part, &part));
  const int parts = parts_of(a, sq), n = sq.nq * a.group, tiles = (n + kFewRows - 1) / kFewRows;
  if (part < 0 || part >= parts || n == 0) return;
  const bool cut = tiles == 1 && parts > 1;
  const int shift = sq.nk - sq.nq;
  const T* K = static_cast<const T*>(a.K) + sq.k0 * a.ldk + (int64_t)kv * hd;
  const T* V = static_cast<const T*>(a.V) + sq.k0 * a.ldv + (int64_t)kv * hd;
  const float c = a.scale * kLog2e;
  const Lane lane_at = R::lane_at();
  float2* const sums = reinterpret_cast<float2*>(a.rows) + part_row(a, slot, kv);
  for (int tile = cut ? 0 : part; tile < tiles; tile += parts) {
    const int row = tile * kFewRows + (lane & 31), i = row / a.group, head = kv * a.group + row % a.group;
    const bool live = row < n;
    // the keys that some row sees, and this workgroup's of them
    const int last = (min((tile + 1) * kFewRows, n) - 1) / a.group;
    int j0 = keys_of(a, tile * kFewRows / a.group + shift, sq.nk).lo, j1 = keys_of(a, last + shift, sq.nk).hi;
    if (cut) {
      const int each = ((sq.nk + parts - 1) / parts + 31) / 32 * 32;  // parts of one length
      j0 = max(j0, part * each);
      j1 = min(j1, part * each + each);
      if (j0 >= j1) {  // none: a part that the join passes over
        if ((int)threadIdx.x < kFewRows) sums[threadIdx.x] = make_float2(-INFINITY, 0.f);
        return;
      }
    }
    Frag<T> q[C / 16];
    row_frags<T, C, HOW>(q, static_cast<const T*>(a.Q) + (sq.q0 + i) * a.ldq + (int64_t)head * hd, live, hd, lane);
    Sees see = live ? keys_of(a, i + shift, sq.nk) : Sees{0, 0};
    see = Sees{max(see.lo, j0), min(see.hi, j1)};
    f32x16_v acc[C / 32] = {};
    float m = -INFINITY, l = 0.f;
    const Span all = keys_of_rows(a, tile * kFewRows / a.group, last, sq);
    // 32 keys from j on, whose K and V lie at lds + t and + v behind it; between() stands between their products
    const auto step = [&](int t, int v, int j, const auto& between) __attribute__((always_inline)) {
      const Lane at = lane_at + t;
      f32x16_v s = {};
#pragma unroll
      for (int kk = 0; kk < C / 16; ++kk)
        if (within<T>(16 * kk, hd)) mma(s, R::along(lds, at, 0, kk), q[kk]);
      if (j + 32 > j1 || !all.all(j, j + 32)) {
        const Sees on = see.from(j);
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = on.has(acc_row(e)) ? s[e] : -INFINITY;
      }
      float top = s[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
      top = max_halves(top);
      if (__any((top - m) * c > kSlack)) {
        const float was = m;
        m = fmaxf(m, top);
        const float keep = exp2_of((was - (m == -INFINITY ? 0.f : m)) * c);
        l *= keep;
#pragma unroll
        for (int d = 0; d < C / 32; ++d) acc[d] *= keep;
      }
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[e] = exp2_of((s[e] - base) * c);
        l += s[e];
      }
      between();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Frag<T> p = to_frag<T>(s, h);
#pragma unroll
        for (int d = 0; d < C / 32; ++d)
          if (within<T>(32 * d, hd)) mma(acc[d], R::across(lds + v, at, 16 * h, 32 * d), p);
      }
    };
    if constexpr (HOW != kStaged) {
      const int mine = wave * 2 * R::bytes(32);
      zero_tail<C>(lds + mine, 64, hd, lane, 64);
      const DmaRows<C, 32, 1, true> dma(0);
      const auto keys = [&](int j) __attribute__((always_inline)) { dma.copy(lds + mine, K, a.ldk, j, sq.nk, hd, 0); };
      const auto values = [&](int j) __attribute__((always_inline)) {
        dma.copy(lds + mine + R::bytes(32), V, a.ldv, j, sq.nk, hd, 0);
      };
      // all of this wave's copies but those of the last 32 rows
      const auto all_but_last = [] __attribute__((always_inline)) {
        if constexpr (R::bytes(32) == 8192) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
        else asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
      };
      static_assert(R::bytes(32) == 8192 || R::bytes(32) == 4096, "1 KB a copy");
      int j = j0 + 32 * wave;
      if (j < j1) {
        keys(j);
        values(j);
      }
      settle<T>(q);
      for (; j < j1; j += KT) {
        const bool more = j + KT < j1;
        all_but_last();
        step(mine, R::bytes(32), j, [&]() __attribute__((always_inline)) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the keys are read
          if (more) {
            keys(j + KT);
            all_but_last();
          } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
          }
        });
        if (more) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the values are read
          values(j + KT);
        }
      }
    } else {
      const auto tile_at = [&](int t, int j) __attribute__((always_inline)) {
        if (j + 32 * wave < j1) step(t + R::bytes(32) * wave, R::bytes(KT), j + 32 * wave, [] {});
      };
      over_tiles<T, C, HOW, KT>(lds, K, a.ldk, V, a.ldv, sq.nk, hd, j0, j1, tile_at);
    }
    l = sum_halves(l);
    // the waves' sums, added in their order: wave w takes columns 32 w and up
    __syncthreads();
    float* mine = reinterpret_cast<float*>(lds) + wave * 64 * (C / 2 + 2) + lane;
#pragma unroll
    for (int d = 0; d < C / 32; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) mine[(16 * d + e) * 64] = acc[d][e];
    mine[(C / 2) * 64] = m;
    mine[(C / 2 + 1) * 64] = l;
    __syncthreads();
    if (wave < C / 32) {
      const float* all = reinterpret_cast<const float*>(lds) + lane;
      float f[kWaves], sum = 0.f;
      m = -INFINITY;
#pragma unroll
      for (int x = 0; x < kWaves; ++x) m = fmaxf(m, f[x] = all[(x * (C / 2 + 2) + C / 2) * 64]);
      f32x16_v o = {};
#pragma unroll
      for (int x = 0; x < kWaves; ++x) {
        f[x] = exp2_of((f[x] - (m == -INFINITY ? 0.f : m)) * c);
        sum += f[x] * all[(x * (C / 2 + 2) + C / 2 + 1) * 64];
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] += f[x] * all[(x * (C / 2 + 2) + 16 * wave + e) * 64];
      }
      if (cut) {
        float* to = a.rows + a.part_head + (part_row(a, slot, kv) + (lane & 31)) * C + 32 * wave + 4 * (lane >> 5);
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<float4*>(to + 8 * g) = make_float4(o[4 * g], o[4 * g + 1], o[4 * g + 2], o[4 * g + 3]);
        if (wave == 0 && lane < 32) sums[lane] = make_float2(m, sum);
      } else if (live) {
        T* out = static_cast<T*>(a.out) + (sq.q0 + i) * a.ldout + (int64_t)head * hd + 32 * wave;
        const f32x16_v columns[1] = {o};
        store_row<T, 32, HOW>(out, columns, sum == 0.f ? 0.f : 1.f / sum, hd - 32 * wave, lane);
        if (wave == 0 && lane < 32)
          a.lse[(int64_t)head * a.q.rows + sq.q0 + i] = sum == 0.f ? -INFINITY : m * a.scale + kLn2 * log2f(sum);
      }
    }
    __syncthreads();  // the next tile's copies
  }
}
// The parts of one query and head, in their order: a wave each.
template <typename T, int C> __global__ __launch_bounds__(kThreads) void k_attn_join(AttnArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t at = a.join0 + (int64_t)blockIdx.x * kWaves + wave_id();
  const int64_t i = at / a.heads;
  const int head = (int)(at % a.heads);
  if (i >= a.q.rows || i < first_row(a.q, 0) || i >= first_row(a.q, a.batch)) return;
  const int s = seq_of_row(a.q, a.batch, i);
  const Seq sq = sequence(a, s);
  const int kv = head / a.group, row = (int)(i - sq.q0) * a.group + head % a.group, parts = parts_of(a, sq);
  if (sq.nq * a.group > kFewRows || parts == 1) return;  // complete
  // offsets that decrease may name a sequence without this row, whose place among the parts would be outside them
  if (i < sq.q0 || i >= sq.q0 + sq.nq) return;
  constexpr int kGroup = 16, E = (C + 63) / 64;
  const int64_t slot = (int64_t)((uint32_t)sq.k0 / (uint32_t)a.part) + s;
  const float c = a.scale * kLog2e;
  const float2* const sums = reinterpret_cast<const float2*>(a.rows);
  float m = -INFINITY, sum = 0.f, o[E] = {};
  for (int x0 = 0; x0 < parts; x0 += kGroup) {
    // 16 parts: their maxima and sums a part a lane, their O a part a register, all on the way together
    const int n = min(parts - x0, kGroup);
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < n) ml = sums[part_row(a, slot + x0 + lane, kv) + row];
    float v[kGroup][E];
#pragma unroll
    for (int x = 0; x < kGroup; ++x)
#pragma unroll
      for (int e = 0; e < E; ++e)
        v[x][e] = a.rows[a.part_head + (part_row(a, slot + x0 + min(x, n - 1), kv) + row) * C +
                         min(64 * e + lane, C - 1)];
    float top = fmaxf(m, ml.x);
#pragma unroll
    for (int d = 1; d < kGroup; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    top = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(top), 0));
    const float base = top == -INFINITY ? 0.f : top, keep = exp2_of((m - base) * c);
    m = top;
    // a part that saw no key has no O: whatever is read there counts 0
    const bool none = ml.x == -INFINITY && ml.y == 0.f;
    const float f = none ? 0.f : exp2_of((ml.x - base) * c);
    sum = sum * keep + f * ml.y;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= keep;
    const uint64_t there = __ballot(!none);
#pragma unroll
    for (int x = 0; x < kGroup; ++x) {
      const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), x));
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += there >> x & 1 ? w * v[x][e] : 0.f;
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  T* out = static_cast<T*>(a.out) + i * a.ldout + (int64_t)head * a.hd;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (64 * e + lane < a.hd) out[64 * e + lane] = from_f32<T>(sum == 0.f ? 0.f : o[e] / sum);
  if (lane == 0) a.lse[(int64_t)head * a.q.rows + i] = sum == 0.f ? -INFINITY : m * a.scale + kLn2 * log2f(sum);
}

// ---- backward --------------------------------------------------------------
// Two launches, which each form S and P again (7 products in place of 5): with one, dQ would be added to by atomics, in an
// order of their own every time, or need a copy for every tile of keys.
//
// dQ of 128 queries of one head.  385 us, 715 TFLOP/s of its three products: the matrix pipe is busy 60%.  It also leaves,
// for the second launch, D = dO . O and the lse as its exponent takes it: in units of log2 for bf16, +infinity for a query
// that sees nothing (p = 2^-infinity).
template <typename T> PX_DEV float prob(float s, float lse, float scale, float c) {
  // fp32 keeps the digits of a difference of logarithms; bf16's p has fewer than one fma leaves
  return sizeof(T) == 4 ? exp2_of((s * scale - lse) * kLog2e) : exp2_of(fmaf(s, c, -lse));
}
template <typename T, int C, int HOW> __global__ __launch_bounds__(kThreads, HOW ? 2 : 1) void k_attn_dq(AttnArgs a) {
  constexpr int KT = kTile<T>, NB = KT / 32, BUFS = HOW ? 2 : 1;
  typedef RowsOf<T, C> R;
  __shared__ __align__(16) char lds[BUFS * 2 * R::bytes(KT)];
  const int lane = threadIdx.x & 63, wave = wave_id(), hd = HOW == kWhole ? C : a.hd;
  const int head = head_of(a, blockIdx.x % a.heads);
  int tile;
  const Seq sq =
      sequence(a, tile_of(a.q, a.batch, a.slots, blockIdx.x / a.heads, kRows, gridDim.x > kAtOnce, true, &tile));
  const int w0 = tile * kRows;
  if (tile < 0 || w0 >= sq.nq) return;
  const int shift = sq.nk - sq.nq, i = w0 + 32 * wave + (lane & 31);
  const bool live = i < sq.nq;
  const int row_hd = HOW == kWhole ? C : a.row_hd;
  const T* K = static_cast<const T*>(a.K) + sq.k0 * a.ldk + (int64_t)(head / a.group) * row_hd;
  const T* V = static_cast<const T*>(a.V) + sq.k0 * a.ldv + (int64_t)(head / a.group) * row_hd;
  Frag<T> q[C / 16], g[C / 16];
  row_frags<T, C, HOW>(q, static_cast<const T*>(a.Q) + (sq.q0 + i) * a.ldq + (int64_t)head * hd, live, hd, lane);
  float delta = 0.f;
  {
    Frag<T> o[C / 16];
    row_frags<T, C, HOW>(g, static_cast<const T*>(a.dO) + (sq.q0 + i) * a.lddo + (int64_t)head * hd, live, hd, lane);
    row_frags<T, C, HOW>(o, static_cast<const T*>(a.O) + (sq.q0 + i) * a.ldo + (int64_t)head * hd, live, hd, lane);
#pragma unroll
    for (int kk = 0; kk < C / 16; ++kk)
#pragma unroll
      for (int e = 0; e < 8; ++e) delta += (float)g[kk][e] * (float)o[kk][e];
  }
  delta = sum_halves(delta);
  const int64_t at = (int64_t)head * a.q.rows + sq.q0 + i;
  float lse = live ? a.lse[at] : -INFINITY;
  const Sees see = live && lse != -INFINITY ? keys_of(a, i + shift, sq.nk) : Sees{0, 0};
  lse = lse == -INFINITY ? INFINITY : sizeof(T) == 4 ? lse : lse * kLog2e;
  if (live && lane < 32) {
    a.rows[at] = lse;
    a.rows[(int64_t)a.heads * a.q.rows + at] = delta;
  }
  const Span w = keys_of_wave(a, w0 + 32 * wave, sq);
  const int last = min(w0 + kRows, sq.nq) - 1;
  const int j0 = keys_of(a, w0 + shift, sq.nk).lo / KT * KT, j1 = keys_of(a, last + shift, sq.nk).hi;
  const float c = a.scale * kLog2e;
  const Lane lane_at = R::lane_at();
  f32x16_v acc[C / 32] = {};
  const auto step = [&](int tile, int j) __attribute__((always_inline)) {
    const Lane at = (lane_at + tile).here();
    const char *const tk = lds, *const tv = lds + R::bytes(KT);
    const bool masked = !w.all(j, j + KT);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      f32x16_v s = {}, dp = {};
#pragma unroll
      for (int kk = 0; kk < C / 16; ++kk) {
        if (!within<T>(16 * kk, hd)) continue;
        mma(s, R::along(tk, at, 32 * b, kk), q[kk]);
        mma(dp, R::along(tv, at, 32 * b, kk), g[kk]);
      }
      if (masked) {
        const uint32_t on = see.from(j + 32 * b).bits();
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = on >> acc_row(e) & 1 ? s[e] : -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = prob<T>(s[e], lse, a.scale, c) * (dp[e] - delta);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Frag<T> p = to_frag<T>(s, h);
#pragma unroll
        for (int d = 0; d < C / 32; ++d)
          if (within<T>(32 * d, hd)) mma(acc[d], R::across(tk, at, 32 * b + 16 * h, 32 * d), p);
        // A tile that a mask cuts is multiplied with what that rounding left too: the queries that see few keys, whose
        // gradients are the largest, have all or most of theirs there.  dQ of 2 x 4096 causal tokens is 2.30e-3 off in
        // the norm (1.66e-3 of it rounding dQ itself) instead of 2.51e-3, for 1% of the time.
        if (sizeof(T) == 2 && masked) {
          const Frag<T> rest = rest_of<T>(s, h, p);
#pragma unroll
          for (int d = 0; d < C / 32; ++d) mma(acc[d], R::across(tk, at, 32 * b + 16 * h, 32 * d), rest);
        }
      }
    }
  };
  over_tiles<T, C, HOW, KT>(lds, K, a.ldk, V, a.ldv, sq.nk, row_hd, j0, j1,
                            [&](int tile, int j) __attribute__((always_inline)) {
                              if (w.any(j, j + KT)) step(tile, j);
                            });
  if (live)
    store_row<T, C, HOW>(static_cast<T*>(a.out) + (sq.q0 + i) * a.ldout + (int64_t)head * hd, acc, a.scale, hd, lane);
}

// dK and dV of 128 keys of one key head: its query heads one after another, so that their sum has one order.  Where that
// gives the card too few workgroups, they share the query heads: each leaves its sums in fp32, and k_attn_dkv_sum adds
// them in the heads' order.  Of a block of 32 queries (`tq`, `tg`: their rows and dO in LDS, `rows` and `deltas`: their lse
// and D), key(kk) and value(kk) are the operands of the wave's keys.
template <typename T, int C, class FK, class FV>
PX_DEV void dkv_block(f32x16_v (&dk)[C / 32], f32x16_v (&dv)[C / 32], const char* tq, const char* tg, const Lane& at,
                      const float* rows, const float* deltas, bool masked, const Sees& see, float scale, float c, int hd,
                      const FK& key, const FV& value) {
  typedef RowsOf<T, C> R;
  f32x16_v s = {}, dp = {};
#pragma unroll
  for (int kk = 0; kk < C / 16; ++kk) {
    if (!within<T>(16 * kk, hd)) continue;
    mma(s, R::along(tq, at, 0, kk), key(kk));
    mma(dp, R::along(tg, at, 0, kk), value(kk));
  }
  if (masked) {
    const uint32_t on = see.bits();
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = on >> acc_row(e) & 1 ? s[e] : -INFINITY;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r = acc_row(4 * u);  // four rows of a lane lie side by side
    const float4 l4 = *reinterpret_cast<const float4*>(rows + r), d4 = *reinterpret_cast<const float4*>(deltas + r);
    const float l[4] = {l4.x, l4.y, l4.z, l4.w}, dl[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int e = 4 * u + x;
      s[e] = prob<T>(s[e], l[x], scale, c);
      dp[e] = s[e] * (dp[e] - dl[x]);
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const Frag<T> p = to_frag<T>(s, x), g = to_frag<T>(dp, x);
#pragma unroll
    for (int d = 0; d < C / 32; ++d) {
      if (!within<T>(32 * d, hd)) continue;
      mma(dv[d], R::across(tg, at, 16 * x, 32 * d), p);
      mma(dk[d], R::across(tq, at, 16 * x, 32 * d), g);
    }
  }
}

// The keys of a workgroup, and the queries that see some of them.
struct KeyTile {
  Seq sq;
  int head, share, w0, shift, i0, i1;  // share: which of the workgroups that share the key head's query heads
  int first, heads;                    // its query heads
  bool any;
};
PX_DEV KeyTile key_tile(const AttnArgs& a, int QT) {
  KeyTile k;
  const int kv_heads = a.heads / a.group;
  k.head = (int)(blockIdx.x % kv_heads);
  k.share = (int)(blockIdx.x / kv_heads % a.shares);
  k.heads = a.group / a.shares;
  k.first = k.head * a.group + k.share * k.heads;
  int tile;
  k.sq = sequence(a, tile_of(a.k, a.batch, a.slots, blockIdx.x / kv_heads / a.shares, kRows, gridDim.x > kAtOnce, false,
                            &tile));
  k.w0 = tile * kRows;
  k.any = tile >= 0 && k.w0 < k.sq.nk;
  k.shift = k.sq.nk - k.sq.nq;
  const int last = min(k.w0 + kRows, k.sq.nk) - 1;
  k.i0 = max(places_of(a, k.w0, k.shift, k.sq.nk).lo - k.shift, 0) / QT * QT;
  k.i1 = places_of(a, last, k.shift, k.sq.nk).hi - k.shift;
  return k;
}
// places that see some, and all, of the 32 keys from `first` on
PX_DEV Span places_of_wave(const AttnArgs& a, int first, const KeyTile& k) {
  const int end = first + 31, nk = k.sq.nk;
  Span w = {{0, 0}, {0, 0}};
  if (first < nk) w.some = Sees{places_of(a, first, k.shift, nk).lo, places_of(a, min(end, nk - 1), k.shift, nk).hi};
  if (end < nk) w.each = Sees{places_of(a, end, k.shift, nk).lo, places_of(a, first, k.shift, nk).hi};
  return w;
}

// a key's row of dK (which = 0) or dV (1), or where this share's goes
template <typename T, int C, int HOW>
PX_DEV void store_grad(const AttnArgs& a, const KeyTile& k, int which, int key, const f32x16_v (&acc)[C / 32], int hd,
                       int lane) {
  if (a.shares == 1) {
    T* out = which ? static_cast<T*>(a.out2) + (k.sq.k0 + key) * a.ldout2
                   : static_cast<T*>(a.out) + (k.sq.k0 + key) * a.ldout;
    store_row<T, C, HOW>(out + (int64_t)k.head * hd, acc, which ? 1.f : a.scale, hd, lane);
  } else {
    const int64_t row = ((int64_t)(2 * k.share + which) * (a.heads / a.group) + k.head) * a.k.rows + k.sq.k0 + key;
    store_row<float, C, kWhole>(a.parts + row * C, acc, which ? 1.f : a.scale, C, lane);
  }
}
template <typename T, int C> __global__ __launch_bounds__(kThreads) void k_attn_dkv_sum(AttnArgs a) {
  const int kv_heads = a.heads / a.group, c = (int)(threadIdx.x % (C / 4)) * 4;
  const int64_t n = (int64_t)blockIdx.x * (kThreads / (C / 4)) + threadIdx.x / (C / 4);  // row and head of both
  const int64_t row = n / kv_heads;
  const int head = (int)(n % kv_heads);
  if (row >= a.k.rows || row < first_row(a.k, 0) || row >= first_row(a.k, a.batch)) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = 0; x < a.shares; ++x) {
      const int64_t at = (((int64_t)(2 * x + which) * kv_heads + head) * a.k.rows + row) * C + c;
      const float4 f = *reinterpret_cast<const float4*>(a.parts + at);
      sum = make_float4(sum.x + f.x, sum.y + f.y, sum.z + f.z, sum.w + f.w);
    }
    T* out = which ? static_cast<T*>(a.out2) + row * a.ldout2 : static_cast<T*>(a.out) + row * a.ldout;
    out += (int64_t)head * a.hd;
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < a.hd) out[c + i] = from_f32<T>(v[i]);
  }
}

// Any type, head and alignment: 4 waves, which hold their keys and values in registers.
template <typename T, int C> __global__ __launch_bounds__(kThreads) void k_attn_dkv(AttnArgs a) {
  constexpr int QT = kTile<T>;
  typedef RowsOf<T, C> R;
  __shared__ __align__(16) char lds[2 * R::bytes(QT)];
  __shared__ float rows[2][QT];  // lse, D
  const int lane = threadIdx.x & 63, wave = wave_id();
  const KeyTile t = key_tile(a, QT);
  if (!t.any) return;
  const Seq& sq = t.sq;
  const int j = t.w0 + 32 * wave + (lane & 31);  // this lane's key
  const bool live = j < sq.nk;
  Frag<T> k[C / 16], v[C / 16];
  row_frags<T, C, kStaged>(k, static_cast<const T*>(a.K) + (sq.k0 + j) * a.ldk + (int64_t)t.head * a.hd, live, a.hd, lane);
  row_frags<T, C, kStaged>(v, static_cast<const T*>(a.V) + (sq.k0 + j) * a.ldv + (int64_t)t.head * a.hd, live, a.hd, lane);
  const Sees see = live ? places_of(a, j, t.shift, sq.nk) : Sees{0, 0};
  const Span w = places_of_wave(a, t.w0 + 32 * wave, t);
  const float c = a.scale * kLog2e;
  const Lane lane_at = R::lane_at();
  f32x16_v dk[C / 32] = {}, dv[C / 32] = {};
  const int64_t more = (int64_t)a.heads * a.q.rows;
  const int per = t.i1 > t.i0 ? (t.i1 - t.i0 + QT - 1) / QT : 0, count = per * t.heads;  // tiles: heads x queries
  Staged<T, C, QT> q, g;
  float row_value = 0.f;  // of the first 2 QT threads: lse, D
  const auto load = [&](int n) __attribute__((always_inline)) {
    const int h = t.first + n / per, i = t.i0 + n % per * QT;
    q.load(static_cast<const T*>(a.Q) + sq.q0 * a.ldq + (int64_t)h * a.hd, a.ldq, i, sq.nq, a.hd);
    g.load(static_cast<const T*>(a.dO) + sq.q0 * a.lddo + (int64_t)h * a.hd, a.lddo, i, sq.nq, a.hd);
    if ((int)threadIdx.x < 2 * QT)
      row_value = a.rows[(int)threadIdx.x / QT * more + (int64_t)h * a.q.rows + sq.q0 +
                         min(i + (int)threadIdx.x % QT, sq.nq - 1)];
  };
  if (count > 0) load(0);
  for (int n = 0; n < count; ++n) {
    const int i = t.i0 + n % per * QT;
    __syncthreads();
    q.put(lds);
    g.put(lds + R::bytes(QT));
    if ((int)threadIdx.x < 2 * QT) rows[0][threadIdx.x] = row_value;
    __syncthreads();
    if (n + 1 < count) load(n + 1);
#pragma unroll
    for (int b = 0; b < QT; b += 32) {
      const int p = i + b + t.shift, r = b + 4 * (lane >> 5);
      if (w.any(p, p + 32))
        dkv_block<T, C>(dk, dv, lds, lds + R::bytes(QT), lane_at + R::bytes(b), rows[0] + r, rows[1] + r,
                               !w.all(p, p + 32), see.from(p), a.scale, c, a.hd, [&](int kk) { return k[kk]; },
                               [&](int kk) { return v[kk]; });
    }
  }
  if (!live) return;
  store_grad<T, C, kStaged>(a, t, 0, j, dk, a.hd, lane);
  store_grad<T, C, kStaged>(a, t, 1, j, dv, a.hd, lane);
}

// By direct copies.  The accumulators of 32 keys take 128 registers; with the keys and values
// beside them a SIMD holds one wave, whose products and exponentials follow each other.  Here they stay in LDS, and 8
// waves take the same 128 keys, four of them the first 32 queries of a tile of 64 and four the others: two waves a SIMD.
// The halves' sums are added at the end, the first one's first.  545 us, 670 TFLOP/s of its four products: the matrix
// pipe is busy 54%, LDS 47%.  One wave a SIMD with keys and values in registers takes 870 us.
template <int C> struct Dkv {
  static constexpr int W = 8, QT = 64;
  // copies that the compiler does not count: 64 columns 564 -> 530 us (2 x 4096, the whole backward), but 96 and 128 are 1%
  // slower with them
  static constexpr bool OWN = C <= 64;
  static constexpr int KEYS = RowsOf<bf16_t, C>::bytes(kRows), TILE = RowsOf<bf16_t, C>::bytes(QT);
  static constexpr int BUF = 2 * TILE + 2 * QT * 4;  // queries, dO, lse, D
  static constexpr int EXCHANGE = W * 64 * (C / 32) * 16 * 4;
  static constexpr int LDS = 2 * KEYS + 2 * BUF > EXCHANGE ? 2 * KEYS + 2 * BUF : EXCHANGE;
};
template <int C, int HOW> __global__ __launch_bounds__(512, 2) void k_attn_dkv_dma(AttnArgs a) {
  typedef bf16_t T;
  typedef RowsOf<T, C> R;
  typedef Dkv<C> P;
  constexpr int QT = P::QT;
  extern __shared__ __align__(16) char lds[];
  char *const tk = lds, *const tv = lds + P::KEYS, *const bufs = lds + 2 * P::KEYS;
  const int lane = threadIdx.x & 63, wave = wave_id(), hd = HOW == kWhole ? C : a.row_hd;
  const int keys = 32 * (wave & 3), half = wave >> 2;
  const KeyTile t = key_tile(a, QT);
  if (!t.any) return;
  const Seq& sq = t.sq;
  const int j = t.w0 + keys + (lane & 31);  // this lane's key
  const bool live = j < sq.nk;
  const Sees see = live ? places_of(a, j, t.shift, sq.nk) : Sees{0, 0};
  const Span w = places_of_wave(a, t.w0 + keys, t);
  const float c = a.scale * kLog2e;
  f32x16_v dk[C / 32] = {}, dv[C / 32] = {};
  const T* Q = static_cast<const T*>(a.Q) + sq.q0 * a.ldq;
  const T* G = static_cast<const T*>(a.dO) + sq.q0 * a.lddo;
  const int64_t at = sq.q0 + (int64_t)t.first * a.q.rows, more = (int64_t)a.heads * a.q.rows;
  const int per = t.i1 > t.i0 ? (t.i1 - t.i0 + QT - 1) / QT : 0, count = per * t.heads;  // tiles: heads x queries
  const DmaRows<C, QT, P::W, P::OWN> dma(wave);
  const auto fetch = [&](char* b, int h, int i) __attribute__((always_inline)) {
    const int64_t col = (int64_t)(t.first + h) * hd;
    dma.copy(b, Q + col, a.ldq, i, sq.nq, hd, wave);
    dma.copy(b + P::TILE, G + col, a.lddo, i, sq.nq, hd, wave);
    if (wave < 2) {  // 64 values each: wave 0 the lse, wave 1 D
      const float* x = a.rows + at + wave * more + (int64_t)h * a.q.rows;
      copy_to_lds<4, P::OWN>(b + 2 * P::TILE + wave * QT * 4, reinterpret_cast<const char*>(x + i),
                     4u * (uint32_t)min(lane, sq.nq - 1 - i));
    }
  };
  const Lane lane_at = R::lane_at();
  const auto compute = [&](int tile, int i) __attribute__((always_inline)) {
    const int p = i + 32 * half + t.shift;
    const float* rows = reinterpret_cast<const float*>(lds + tile + 2 * P::TILE) + 32 * half + 4 * (lane >> 5);
    const Lane at = (lane_at + (tile + R::bytes(32 * half))).here(), keys_at = (lane_at + R::bytes(keys)).here();
    if (w.any(p, p + 32))
      dkv_block<T, C>(dk, dv, lds, lds + P::TILE, at, rows, rows + QT, !w.all(p, p + 32), see.from(p), a.scale, c, hd,
                      [&](int kk) { return R::along(tk, keys_at, 0, kk); },
                      [&](int kk) { return R::along(tv, keys_at, 0, kk); });
  };
  if (count > 0) {
    const DmaRows<C, kRows, P::W, P::OWN> whole(wave);
    whole.copy(tk, static_cast<const T*>(a.K) + sq.k0 * a.ldk + (int64_t)t.head * hd, a.ldk, t.w0, sq.nk, hd, wave);
    whole.copy(tv, static_cast<const T*>(a.V) + sq.k0 * a.ldv + (int64_t)t.head * hd, a.ldv, t.w0, sq.nk, hd, wave);
    fetch(bufs, 0, t.i0);
    zero_tail<C>(tk, 2 * kRows, hd, (int)threadIdx.x, 64 * P::W);
    for (int b = 0; b < 2; ++b) zero_tail<C>(bufs + b * P::BUF, 2 * QT, hd, (int)threadIdx.x, 64 * P::W);
  }
  int h = 0, i = t.i0;
  for (int n = 0, buf = 0; n < count; ++n, buf ^= P::BUF) {
    copies_done();
    __syncthreads();  // this tile is there, and the other buffer is done with
    const int now = i;
    i += QT;
    if (i >= t.i1) i = t.i0, ++h;
    if (n + 1 < count) fetch(bufs + (buf ^ P::BUF), h, i);
    compute(2 * P::KEYS + buf, now);
  }
  // the waves of the first queries take the others' dK, those of the others the first ones' dV
  __syncthreads();
  float* mine = reinterpret_cast<float*>(lds) + wave * 64 * (C / 2) + lane;
  const float* other = reinterpret_cast<const float*>(lds) + (wave ^ 4) * 64 * (C / 2) + lane;
#pragma unroll
  for (int d = 0; d < C / 32; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) mine[(16 * d + e) * 64] = half ? dk[d][e] : dv[d][e];
  __syncthreads();
#pragma unroll
  for (int d = 0; d < C / 32; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float x = other[(16 * d + e) * 64];
      dk[d][e] = half ? x + dv[d][e] : dk[d][e] + x;
    }
  if (!live) return;
  store_grad<T, C, HOW>(a, t, half, j, dk, HOW == kWhole ? C : a.hd, lane);
}

// Rows of heads of any length as rows of heads of a multiple of 8 columns, zeros behind the head: 16 bytes a thread.
struct Pack {
  const void* from[4];
  bf16_t* to[4];
  int64_t ld[4];
  Side side[4];
  int heads[4];
  int batch, hd, row_hd;
};
__global__ __launch_bounds__(kThreads) void k_attn_pack(Pack a) {
  const int m = blockIdx.y, k = a.row_hd / 8, per = a.heads[m] * k;
  const int64_t end = first_row(a.side[m], a.batch) * per;
  for (int64_t x = first_row(a.side[m], 0) * per + (int64_t)blockIdx.x * kThreads + threadIdx.x; x < end;
       x += (int64_t)gridDim.x * kThreads) {
    const int64_t row = x / per;
    const int head = (int)(x - row * per) / k, c = (int)(x - row * per) % k;
    bf16_t v[8];
    load8<kStaged>(v, static_cast<const bf16_t*>(a.from[m]) + row * a.ld[m] + (int64_t)head * a.hd, true, 8 * c, a.hd);
    __builtin_memcpy(a.to[m] + 8 * x, v, sizeof(v));
  }
}

int64_t slots_of(int64_t rows, int batch, int R = kRows) { return rows / R + batch; }

AttnArgs args_of(const AttnDesc& d) {
  AttnArgs a = {};
  a.q = Side{d.cu_q, d.Tq, d.Tq / d.batch};
  a.k = Side{d.cu_k, d.Tk, d.Tk / d.batch};
  a.batch = d.batch;
  a.heads = d.heads;
  a.group = d.heads / d.kv_heads;
  a.hd = a.row_hd = d.hd;
  a.window = d.window;
  a.causal = d.causal;
  a.scale = d.scale;
  return a;
}

// columns that the kernels are built for
int width(const AttnDesc& d) { return (int)round_up(d.hd, d.dt == BF16 ? 32 : 64); }
// f(T(), std::integral_constant<int, C>()) for the type and the width
template <class F> void pick(const AttnDesc& d, F&& f) {
  const int c = width(d);
  if (d.dt == BF16) {
    if (c == 32) f(bf16_t(), std::integral_constant<int, 32>());
    else if (c == 64) f(bf16_t(), std::integral_constant<int, 64>());
    else if (c == 96) f(bf16_t(), std::integral_constant<int, 96>());
    else f(bf16_t(), std::integral_constant<int, 128>());
  } else {
    if (c == 64) f(float(), std::integral_constant<int, 64>());
    else f(float(), std::integral_constant<int, 128>());
  }
}

// whether the direct-to-LDS copies take these heads, and these rows
bool direct_heads(const AttnDesc& d) { return d.dt == BF16 && d.hd % 8 == 0; }
bool direct_rows(const AttnMat& m) {
  return reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && m.ld % 8 == 0 && m.ld <= kDmaLd;
}
// f(std::integral_constant<int, HOW>()), direct: they take both
template <typename T, int C, class F> void pick_how(const AttnDesc& d, bool direct, F&& f) {
  if constexpr (sizeof(T) == 2) {
    if constexpr (C % 64 == 0)
      if (direct && d.hd == C) return f(std::integral_constant<int, kWhole>());
    if (direct) return f(std::integral_constant<int, kDirect>());
  }
  f(std::integral_constant<int, kStaged>());
}

// bf16 heads of no multiple of 8 columns: whether they are laid out as heads of one first, for the direct copies.  It is a
// launch more, which sequences of 128 keys on the average make up for.  75 columns, 8 heads over 4, us through registers
// and laid out first: forward 10.6 and 13.4 at 64 tokens, 19.1 and 15.5 at 256, 51 and 28 at 1024; backward 28.4 and 28.2,
// 54 and 39, 143 and 78; 2 x 4096 tokens of 32 heads forward 512 and 268, backward 2380 and 870.
bool packs(const AttnDesc& d) { return d.dt == BF16 && d.hd % 8 != 0 && d.Tk >= 128 * (int64_t)d.batch; }
int64_t packed_row(const AttnDesc& d, int heads) { return heads * round_up(d.hd, 8); }
size_t packed_bytes(const AttnDesc& d, int64_t rows, int heads) {
  return (size_t)round_up(rows * packed_row(d, heads) * 2, 256);
}
// `mats` (of the queries or of the keys) laid out at ws, where they are from then on
void pack(const AttnDesc& d, AttnArgs& a, AttnMat* const* mats, const bool* keys, int count, void* ws, hipStream_t s) {
  Pack p = {};
  p.batch = d.batch, p.hd = d.hd, p.row_hd = a.row_hd = (int)round_up(d.hd, 8);
  char* to = static_cast<char*>(ws);
  int64_t most = 0;
  for (int i = 0; i < count; ++i) {
    const int heads = keys[i] ? d.kv_heads : d.heads;
    p.side[i] = keys[i] ? a.k : a.q;
    p.from[i] = mats[i]->p, p.ld[i] = mats[i]->ld, p.heads[i] = heads, p.to[i] = reinterpret_cast<bf16_t*>(to);
    *mats[i] = AttnMat{to, packed_row(d, heads)};
    to += packed_bytes(d, p.side[i].rows, heads);
    most = std::max(most, p.side[i].rows * packed_row(d, heads) / 8);
  }
  const unsigned grid = (unsigned)std::min<int64_t>((most + kThreads - 1) / kThreads, 1 << 14);
  if (grid) k_attn_pack<<<dim3(grid, count), kThreads, 0, s>>>(p);
}

// The keys of a workgroup in the forward of few rows; 0 where a tile of 32 rows does not hold a sequence's queries on the
// average, and the tiles of 128 queries are taken (16 tokens over 1 to 8192 keys: 732 us with those).  The average is the
// call's, since the host knows no length: a prompt among single tokens goes the way of the most (128 tokens over 4096 keys
// each, 444 us, with a prompt of 900, 27 us, take 1430 us in one call).  Parts are as long as leaves the card some 512
// workgroups (256 to 1024 measured the same or slower; heads of 128 columns run them in two turns), and a sequence two.
int few_part(const AttnDesc& d) {
  if (d.Tq * (d.heads / d.kv_heads) > (int64_t)kFewRows * d.batch) return 0;
  return (int)std::max<int64_t>(256, round_up(std::min(d.Tk * d.kv_heads / 512, d.Tk / (2 * d.batch)), kFewKeys));
}

// How many workgroups share the query heads of a key head in dK and dV: the fewest that divide them and give two
// workgroups a CU, which their unequal work (causal keys) needs: the backward of 1 x 2048 tokens 303 -> 185 us (fp32 2.63
// -> 1.08 ms) against one; with targets of 256 or 1024 workgroups it was slower.
int key_shares(const AttnDesc& d) {
  const int group = d.heads / d.kv_heads;
  const int64_t grid = slots_of(d.Tk, d.batch) * d.kv_heads;
  int n = 1;
  while (n < group && (group % n || grid * n < 512)) ++n;
  return n;
}

}  // namespace

namespace pxk {

bool attn_fits(const AttnDesc& d) {
  const int64_t most = (int64_t(1) << 23) - 1;  // 512 threads each, and a launch has fewer than 2^32
  return slots_of(d.Tq, d.batch) * d.heads <= most && slots_of(d.Tk, d.batch) * d.kv_heads <= most;
}

size_t attn_fwd_ws_bytes(const AttnDesc& d) {
  const int part = few_part(d);
  if (part == 0 && packs(d)) return 2 * packed_bytes(d, d.Tk, d.kv_heads);
  if (part == 0 || d.Tk <= part) return 0;  // the latter: no sequence has two parts
  return (size_t)slots_of(d.Tk, d.batch, part) * d.kv_heads * kFewRows * (2 + width(d)) * 4;
}
static size_t shares_at(const AttnDesc& d) { return (size_t)round_up((int64_t)d.heads * d.Tq * 8, 256); }
static size_t packed_at(const AttnDesc& d) {
  const int n = key_shares(d);
  return shares_at(d) + (n > 1 ? (size_t)round_up((int64_t)n * 2 * d.kv_heads * d.Tk * width(d) * 4, 256) : 0);
}
size_t attn_bwd_ws_bytes(const AttnDesc& d) {
  return packed_at(d) + (packs(d) ? 2 * packed_bytes(d, d.Tk, d.kv_heads) + 2 * packed_bytes(d, d.Tq, d.heads) : 0);
}

hipError_t attn_fwd(const AttnDesc& d, const AttnMat& Q, const AttnMat& K0, const AttnMat& V0, void* O, int64_t ldo,
                    float* lse, void* ws, hipStream_t s) {
  if (d.Tq == 0) return hipSuccess;
  AttnArgs a = args_of(d);
  AttnMat K = K0, V = V0;
  const bool packed = few_part(d) == 0 && packs(d);
  if (packed) {
    AttnMat* const mats[] = {&K, &V};
    const bool keys[] = {true, true};
    pack(d, a, mats, keys, 2, ws, s);
  }
  a.Q = Q.p, a.ldq = Q.ld, a.K = K.p, a.ldk = K.ld, a.V = V.p, a.ldv = V.ld;
  a.out = O, a.ldout = ldo, a.lse = lse, a.rows = static_cast<float*>(ws);
  a.part = few_part(d);
  const bool direct = packed || (direct_heads(d) && direct_rows(K) && direct_rows(V));
  if (a.part) {
    hipError_t e = hipSuccess;
    const int64_t slots = slots_of(d.Tk, d.batch, a.part);
    a.part_head = 2 * slots * d.kv_heads * kFewRows;
    pick(d, [&](auto t, auto columns) {
      typedef decltype(t) T;
      constexpr int C = decltype(columns)::value;
      pick_how<T, C>(d, direct, [&](auto how) {
        constexpr int HOW = decltype(how)::value, kLds = Few<T, C>::LDS;
        e = px::lds_once<k_attn_few<T, C, HOW>>(kLds);
        if (e == hipSuccess)
          k_attn_few<T, C, HOW><<<dim3((unsigned)(slots * d.kv_heads)), kThreads, kLds, s>>>(a);
      });
      const int64_t rows = d.Tq * d.heads, most = int64_t(1) << 24;  // of a launch, 64 threads each
      for (a.join0 = 0; e == hipSuccess && d.Tk > a.part && a.join0 < rows; a.join0 += most)
        k_attn_join<T, C>
            <<<dim3(px::cdiv(std::min(most, rows - a.join0), kWaves)), kThreads, 0, s>>>(a);
    });
    return e != hipSuccess ? e : hipGetLastError();
  }
  a.slots = slots_of(d.Tq, d.batch);
  pick(d, [&](auto t, auto columns) {
    typedef decltype(t) T;
    constexpr int C = decltype(columns)::value;
    pick_how<T, C>(d, direct, [&](auto how) {
      k_attn_fwd<T, C, decltype(how)::value>
          <<<dim3((unsigned)(a.slots * d.heads)), kThreads * kFwdGroups<T>, 0, s>>>(a);
    });
  });
  return hipGetLastError();
}

hipError_t attn_bwd(const AttnDesc& d, const AttnMat& dO0, const AttnMat& Q0, const AttnMat& K0, const AttnMat& V0,
                    const AttnMat& O, const float* lse, void* dQ, int64_t lddq, void* dK, int64_t lddk, void* dV,
                    int64_t lddv, void* ws, hipStream_t s) {
  AttnArgs a = args_of(d);
  AttnMat dO = dO0, Q = Q0, K = K0, V = V0;
  const bool packed = packs(d);
  if (packed) {
    AttnMat* const mats[] = {&K, &V, &Q, &dO};
    const bool keys[] = {true, true, false, false};
    pack(d, a, mats, keys, 4, static_cast<char*>(ws) + packed_at(d), s);
  }
  const bool direct = packed || (direct_heads(d) && direct_rows(K) && direct_rows(V));
  // dQ reads the caller's rows of Q and dO, dK and dV the ones for the copies
  a.Q = Q0.p, a.ldq = Q0.ld, a.K = K.p, a.ldk = K.ld, a.V = V.p, a.ldv = V.ld, a.O = O.p, a.ldo = O.ld;
  a.dO = dO0.p, a.lddo = dO0.ld;
  a.lse = const_cast<float*>(lse), a.rows = static_cast<float*>(ws);
  if (d.Tq > 0) {
    a.out = dQ, a.ldout = lddq;
    a.slots = slots_of(d.Tq, d.batch);
    pick(d, [&](auto t, auto columns) {
      typedef decltype(t) T;
      constexpr int C = decltype(columns)::value;
      pick_how<T, C>(d, direct, [&](auto how) {
        k_attn_dq<T, C, decltype(how)::value><<<dim3((unsigned)(a.slots * d.heads)), kThreads, 0, s>>>(a);
      });
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (d.Tk == 0) return hipSuccess;
  a.out = dK, a.ldout = lddk, a.out2 = dV, a.ldout2 = lddv;
  a.Q = Q.p, a.ldq = Q.ld, a.dO = dO.p, a.lddo = dO.ld;
  a.shares = key_shares(d);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + shares_at(d));
  a.slots = slots_of(d.Tk, d.batch);
  hipError_t e = hipSuccess;
  pick(d, [&](auto t, auto columns) {
    typedef decltype(t) T;
    constexpr int C = decltype(columns)::value;
    const dim3 grid((unsigned)(a.slots * d.kv_heads * a.shares));
    pick_how<T, C>(d, direct && direct_rows(Q) && direct_rows(dO), [&](auto how) {
      constexpr int HOW = decltype(how)::value;
      if constexpr (HOW == kStaged) {
        k_attn_dkv<T, C><<<grid, kThreads, 0, s>>>(a);
      } else {
        e = px::lds_once<k_attn_dkv_dma<C, HOW>>(Dkv<C>::LDS);
        if (e == hipSuccess) k_attn_dkv_dma<C, HOW><<<grid, 64 * Dkv<C>::W, Dkv<C>::LDS, s>>>(a);
      }
    });
    const int rows = kThreads / (C / 4);  // of a workgroup
    if (e == hipSuccess && a.shares > 1)
      k_attn_dkv_sum<T, C><<<dim3(px::cdiv(d.Tk * d.kv_heads, rows)), rows * (C / 4), 0, s>>>(a);
  });
  return e != hipSuccess ? e : hipGetLastError();
}

}  // namespace pxk
