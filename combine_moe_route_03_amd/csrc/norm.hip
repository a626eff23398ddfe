// norm.hip -- the root-mean-square norm ahead of the router, with the residual's
// addition and an 8-bit copy of its rows, and the quantisation of rows to 8-bit
// integers (quant_int8.h; the blocks of e4m3 are those of quant.h).
//
//   t = round(x + r),  y = t w / sqrt(mean(t^2) + eps),  q, scale from y unrounded
//
// Sums, norms and quotients are held in 64 bits: v_fma_f64 issues at the rate of
// v_fma_f32 here, so that costs nothing next to the bytes, and a value next to the
// border between two integers lands on its own side.
//
// Bound by HBM bytes: every element is read once and kept in registers between the
// row's reduction and the outputs. Norm of 16384 x 7168 bf16 with the residual, y and int8 rows
// out: 173-176 us, 6.0-6.1 TB/s; 45056 x 4096 bf16 to int8: 86 us, 6.4 TB/s. One row of 4096:
// 3.7 us in a graph, latency. Norms of rows wider than 32768 do not fit the 128 registers of a
// block of 1024 threads and keep part of a row in scratch memory (512 rows of 65536, int8 rows
// out: bf16 78 us, 3.9 TB/s; fp32 229 us, 2.5 TB/s).
#include <type_traits>

#include "device.h"
#include "ffn_device.h"
#include "launch.h"
#include "quant.h"
#include "quant_int8.h"

namespace moe {
namespace {

constexpr int kPackThreads = 256;  // block of rows that fit a wave or part of one

// 16 bytes of a row: 8 bf16 or 4 fp32 elements.
template <bool kBF16>
struct RowVec {
  static constexpr int N = kBF16 ? 8 : 4;
  v4u v;
  __device__ __forceinline__ float get(int i) const {
    if constexpr (kBF16) return (i & 1) ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1]);
    else return __uint_as_float(v[i]);
  }
};

template <bool kBF16>
__device__ __forceinline__ v4u pack_row(const float (&f)[RowVec<kBF16>::N]) {
  if constexpr (kBF16)
    return v4u{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
               bf16x2_rne(f[6], f[7])};
  else
    return v4u{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
               __float_as_uint(f[3])};
}

// v in fp32 for one more rounding to a type of 9 significant bits or less, whose result is then
// that of one rounding from 64 bits: where anything lies below the 11th bit, that bit is set and
// the 10 below it are cleared, so that fp32 cannot round the rest onto the border between two
// values. (From 2^-139 on 11 bits are whole steps of fp32; what is less is zero in bf16.) Four
// instructions on the high word: the norm of 16384 x 7168 bf16, int8 rows out, 173 -> 174 us, e4m3
// rows 175 -> 176.5; 512 rows of 65536 77 -> 78 (with fp32 first and a branch for values on a
// border 83).
__device__ __forceinline__ float narrow(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)u, hi = (uint32_t)(u >> 32);
  const uint32_t odd = (lo | (hi & 0x3FFu)) ? ((hi & ~0x3FFu) | 0x400u) : hi;
  return (float)__longlong_as_double((long long)((uint64_t)odd << 32 | lo));
}

template <bool kCache>
__device__ __forceinline__ void put(v4u* p, v4u v) {
  if constexpr (kCache) *p = v;
  else store_stream(p, v);
}
template <bool kCache, int N>
__device__ __forceinline__ void put_q(uint8_t* p, const uint32_t (&w)[N]) {
  typedef uint32_t v2u __attribute__((ext_vector_type(2)));
  if constexpr (N == 2) {
    if constexpr (kCache) *reinterpret_cast<v2u*>(p) = v2u{w[0], w[1]};
    else __builtin_nontemporal_store(v2u{w[0], w[1]}, reinterpret_cast<v2u*>(p));
  } else {
    if constexpr (kCache) *reinterpret_cast<uint32_t*>(p) = w[0];
    else __builtin_nontemporal_store(w[0], reinterpret_cast<uint32_t*>(p));
  }
}

struct Sum {
  __device__ __forceinline__ double operator()(double a, double b) const { return a + b; }
};
struct Max {  // a NaN gives way to a number
  __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};
struct MaxOrNaN {  // of magnitudes, whose order is that of their bits, NaN the largest
  __device__ __forceinline__ double operator()(double a, double b) const {
    return __double_as_longlong(a) > __double_as_longlong(b) ? a : b;
  }
};

// Where a thread stands: a row of L lanes is G of them in one wave (G < 64: several
// rows a wave, or a wave alone), or the whole block (G = 0).
template <int G>
struct Place {
  uint32_t row;    // past the last one: nothing of it is loaded or stored
  uint32_t lane;   // in the row
  uint32_t lanes;  // of the row
  __device__ __forceinline__ Place() {
    if constexpr (G > 0) {
      row = blockIdx.x * (uint32_t)(kPackThreads / G) + threadIdx.x / G;
      lane = threadIdx.x % G;
      lanes = G;
    } else {
      row = blockIdx.x;
      lane = threadIdx.x;
      lanes = blockDim.x;
    }
  }
};

// Reductions over the lanes of a row, each of two values at a time; `part`: kMaxWaves
// places that no other reduction of the kernel uses.
constexpr int kMaxWaves = 16;
template <typename A, typename B>
struct Two {
  A a;
  B b;
};
template <int G, typename A, typename B, typename OpA, typename OpB>
__device__ __forceinline__ Two<A, B> row_reduce(A a, B b, Two<A, B>* part, OpA op_a, OpB op_b) {
  a = group_reduce(a, G > 0 ? G : kWave, op_a);
  b = group_reduce(b, G > 0 ? G : kWave, op_b);
  if constexpr (G > 0) return {a, b};
  if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = {a, b};
  __syncthreads();
  Two<A, B> v = part[0];
  for (uint32_t w = 1; w < blockDim.x / kWave; ++w) v = {op_a(v.a, part[w].a), op_b(v.b, part[w].b)};
  return v;
}

constexpr int kNoQ = 0, kInt8 = 1, kE4M3 = 2;

// One row of G lanes or of a block, P 16-byte vectors a lane. total and y may each be the
// buffer of x or of the residual (not both the same): a lane writes only what it has read.
template <bool kBF16, int kQ, int G, int P, bool kCache>
__global__ __launch_bounds__(G ? kPackThreads : 1024) void add_rms_norm_kernel(
    const v4u* x, const v4u* residual, const v4u* __restrict__ weight, double eps, uint32_t rows,
    uint32_t nvec, v4u* total, v4u* y, uint8_t* __restrict__ q, float* __restrict__ scale) {
  typedef RowVec<kBF16> Vec;
  constexpr int N = Vec::N;
  __shared__ Two<double, double> sums[kMaxWaves], finite[kMaxWaves];
  const Place<G> at;
  const bool live = at.row < rows;
  const size_t base = (size_t)at.row * nvec;
  const double inf = __builtin_huge_val();
  Vec t[P], w[P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const uint32_t c = j * at.lanes + at.lane;
    t[j].v = v4u{0, 0, 0, 0};
    w[j].v = v4u{0, 0, 0, 0};
    if (live && c < nvec) {
      t[j].v = load_stream(x + base + c);
      w[j].v = weight[c];
    }
  }
  if (residual) {
    Vec r[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const uint32_t c = j * at.lanes + at.lane;
      r[j].v = v4u{0, 0, 0, 0};
      if (live && c < nvec) r[j].v = load_stream(residual + base + c);
    }
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const uint32_t c = j * at.lanes + at.lane;
      float f[N];
      // bf16: the fp32 sum is exact or too far below a border to move the rounding
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = t[j].get(i) + r[j].get(i);
      t[j].v = pack_row<kBF16>(f);
      if (live && c < nvec) put<kCache>(total + base + c, t[j].v);
    }
  }
  // the sum of squares, and for integers the largest |t w| (NaN if there is one): y is that
  // times one factor, so its largest value needs no second reduction
  double ss = 0, top = 0;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < P; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const double v = t[j].get(i);
      ss = __builtin_fma(v, v, ss);
      if constexpr (kQ == kInt8) {
        const double u = v * (double)w[j].get(i);
        top = fmax(top, fabs(u));
        nan |= u != u;
      }
    }
  if (nan) top = __builtin_nan("");
  const Two<double, double> all = row_reduce<G>(ss, top, sums, Sum(), MaxOrNaN());
  ss = all.a;
  top = all.b;
  const double r = 1.0 / sqrt(ss / (double)(nvec * N) + eps);
  double inv = 0, most = 0;  // of int8: 1 / scale, 127 scale
  if constexpr (kQ == kInt8) {
    if (__any(top == inf)) {  // the largest finite one (a row of a block: all its waves are here)
      double m = 0;
#pragma unroll
      for (int j = 0; j < P; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const double u = fabs((double)t[j].get(i) * (double)w[j].get(i));
          m = u < inf ? fmax(m, u) : m;
        }
      m = row_reduce<G>(m, 0.0, finite, Max(), Max()).a;
      // an infinite t: its y is infinity times zero
      top = top != inf ? top : (r == 0.0 ? __builtin_nan("") : m);
    }
    top *= r;
    nan = top != top;
    const float s = int8_scale(top);
    inv = nan ? 0.0 : 1.0 / (double)s;
    most = 127.0 * s;
    if (live && at.lane == 0) scale[at.row] = nan ? __builtin_nanf("") : s;
  }
  constexpr uint32_t kGroup = kQuantBlock / N;  // lanes of an e4m3 scale
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const uint32_t c = j * at.lanes + at.lane;
    const bool ok = live && c < nvec;
    double v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (double)t[j].get(i) * (double)w[j].get(i) * r;
    float n[N];  // for bf16 and e4m3
#pragma unroll
    for (int i = 0; i < N; ++i) n[i] = narrow(v[i]);
    if (y && ok) {
      float f[N];
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = kBF16 ? n[i] : (float)v[i];
      put<kCache>(y + base + c, pack_row<kBF16>(f));
    }
    if constexpr (kQ == kInt8) {
      uint32_t o[N / 4];
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        int b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = int8_round(fmin(fmax(v[4 * i + k], -most), most), inv);
        o[i] = pack_int8(b[0], b[1], b[2], b[3]);
      }
      if (ok) put_q<kCache>(q + (base + c) * N, o);
    }
    if constexpr (kQ == kE4M3) {
      double m = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) m = fmax(m, fabs(v[i]));
      if (__any(m == inf)) {
        m = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) m = fabs(v[i]) < inf ? fmax(m, fabs(v[i])) : m;
      }
      m = group_reduce(m, kGroup, Max());
      const int p = scale_exponent(m);
      float f = 1.0f;
      if (__any(p > 118)) {  // y may be past the range of fp32
        const double d = __longlong_as_double((long long)(1023 - p) << 52);  // 2^-p
#pragma unroll
        for (int i = 0; i < N; ++i) n[i] = narrow(v[i] * d);
      } else {
        f = power_of_two(-p);  // n 2^-p is exact, or too small for e4m3
      }
      uint32_t o[N / 4];
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        o[i] = e4m3x4(e4m3_clamp(n[4 * i] * f), e4m3_clamp(n[4 * i + 1] * f),
                      e4m3_clamp(n[4 * i + 2] * f), e4m3_clamp(n[4 * i + 3] * f));
      if (ok) {
        put_q<kCache>(q + (base + c) * N, o);
        const uint32_t groups = (nvec + kGroup - 1) / kGroup;
        if (c % kGroup == 0) scale[(size_t)at.row * groups + c / kGroup] = power_of_two(p);
      }
    }
  }
}

// Rows to int8: the layout of the norm's kernel.
template <bool kBF16, int G, int P, bool kCache>
__global__ __launch_bounds__(G ? kPackThreads : 1024) void quantize_int8_kernel(
    const v4u* __restrict__ x, uint32_t rows, uint32_t nvec, uint8_t* __restrict__ q,
    float* __restrict__ scale) {
  typedef RowVec<kBF16> Vec;
  constexpr int N = Vec::N;
  __shared__ Two<uint32_t, uint32_t> tops[kMaxWaves];
  const Place<G> at;
  const bool live = at.row < rows;
  const size_t base = (size_t)at.row * nvec;
  Vec t[P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const uint32_t c = j * at.lanes + at.lane;
    t[j].v = v4u{0, 0, 0, 0};
    if (live && c < nvec) t[j].v = load_stream(x + base + c);
  }
  uint32_t top = 0, all = 0;  // magnitudes as bits: of the finite values, of all
#pragma unroll
  for (int j = 0; j < P; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t u = __float_as_uint(t[j].get(i)) & 0x7FFFFFFFu;
      const uint32_t f = u < kInfBits ? u : 0u;
      top = f > top ? f : top;
      all = u > all ? u : all;
    }
  const Two<uint32_t, uint32_t> row = row_reduce<G>(all, top, tops, Max(), Max());
  const Int8Row how = int8_row(row.a, row.b);
  if (live && at.lane == 0) scale[at.row] = how.scale;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const uint32_t c = j * at.lanes + at.lane;
    uint32_t o[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      int b[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) b[k] = how.round(t[j].get(4 * i + k));
      o[i] = pack_int8(b[0], b[1], b[2], b[3]);
    }
    if (live && c < nvec) put_q<kCache>(q + (base + c) * N, o);
  }
}

// Lanes and vectors a lane of a row: f(G, P, block, rows a block). Many rows take a wave
// each, up to eight vectors a lane, or else blocks of four vectors a lane: with a vector a
// lane, and so a block of many waves a row, the barriers of the reduction leave the memory
// idle (when that was measured, 45056 rows of 4096 bf16 to int8 151 against 96 us, norm of
// 16384 rows of 7168 207 against 178). Few rows take as many lanes as they have vectors,
// since they are bound by latency, but for more than 512 lanes, which take longer to begin
// (1 row of 7168 5.1 against 4.3 us, 512 rows 11 against 9).
template <bool kBF16, typename F>
hipError_t by_row(uint32_t rows, uint32_t nvec, const F& f) {
  constexpr int kPart = kBF16 ? 16 : 32;  // lanes of 128 columns
  using std::integral_constant;
  const auto go = [&](auto g, auto p, uint32_t block, uint32_t per) {
    return f(g, p, dim3(block), per);
  };
#define MOE_ROW(G, P, BLOCK, PER) \
  return go(integral_constant<int, G>{}, integral_constant<int, P>{}, BLOCK, PER)
  const auto threads = [&](uint32_t p) { return (nvec + p * kWave - 1) / (p * kWave) * kWave; };
  if (nvec <= kPart) MOE_ROW(kPart, 1, kPackThreads, kPackThreads / kPart);
  if (nvec <= kWave) MOE_ROW(kWave, 1, kPackThreads, kPackThreads / kWave);
  if (rows >= 1024) {
    if (nvec <= 2 * kWave) MOE_ROW(kWave, 2, kPackThreads, kPackThreads / kWave);
    if (nvec <= 4 * kWave) MOE_ROW(kWave, 4, kPackThreads, kPackThreads / kWave);
    if (nvec <= 6 * kWave) MOE_ROW(kWave, 6, kPackThreads, kPackThreads / kWave);
    if (nvec <= 8 * kWave) MOE_ROW(kWave, 8, kPackThreads, kPackThreads / kWave);
  } else if (threads(1) <= 512) {
    MOE_ROW(0, 1, threads(1), 1);
  }
  if (threads(4) <= 1024) MOE_ROW(0, 4, threads(4), 1);
  if (threads(8) <= 1024) MOE_ROW(0, 8, threads(8), 1);
  if constexpr (!kBF16) MOE_ROW(0, 16, threads(16), 1);
  return hipErrorInvalidValue;
#undef MOE_ROW
}

template <bool kBF16>
hipError_t norm(int q_format, const void* x, const void* residual, const void* weight, double eps,
                uint32_t rows, uint32_t H, void* total, void* y, void* q, float* scale,
                hipStream_t s) {
  const uint32_t nvec = H / RowVec<kBF16>::N;
  const bool cache = int64_t(rows) * H * (kBF16 ? 2 : 4) <= kCacheReuseBytes;
  return by_row<kBF16>(rows, nvec, [&](auto g, auto p, dim3 block, uint32_t per) {
    constexpr int G = decltype(g)::value, P = decltype(p)::value;
    const auto run = [&](auto kernel) {
      return launch(kernel, dim3((rows + per - 1) / per), block, 0, s, static_cast<const v4u*>(x),
                    static_cast<const v4u*>(residual), static_cast<const v4u*>(weight), eps, rows,
                    nvec, static_cast<v4u*>(total), static_cast<v4u*>(y),
                    static_cast<uint8_t*>(q), scale);
    };
    const auto of = [&](auto c) {
      constexpr bool C = decltype(c)::value;
      return q_format == kInt8   ? run(add_rms_norm_kernel<kBF16, kInt8, G, P, C>)
             : q_format == kE4M3 ? run(add_rms_norm_kernel<kBF16, kE4M3, G, P, C>)
                                 : run(add_rms_norm_kernel<kBF16, kNoQ, G, P, C>);
    };
    return cache ? of(std::true_type{}) : of(std::false_type{});
  });
}

template <bool kBF16>
hipError_t rows_to_int8(const void* x, uint32_t rows, uint32_t cols, void* q, float* scale,
                        hipStream_t s) {
  const uint32_t nvec = cols / RowVec<kBF16>::N;
  const bool cache = int64_t(rows) * cols <= kCacheReuseBytes;
  return by_row<kBF16>(rows, nvec, [&](auto g, auto p, dim3 block, uint32_t per) {
    constexpr int G = decltype(g)::value, P = decltype(p)::value;
    const auto run = [&](auto kernel) {
      return launch(kernel, dim3((rows + per - 1) / per), block, 0, s, static_cast<const v4u*>(x),
                    rows, nvec, static_cast<uint8_t*>(q), scale);
    };
    return cache ? run(quantize_int8_kernel<kBF16, G, P, true>)
                 : run(quantize_int8_kernel<kBF16, G, P, false>);
  });
}

}  // namespace

hipError_t launch_add_rms_norm(int dtype, int q_dtype, int T, int H, const void* x,
                               const void* residual, const void* weight, double eps, void* total,
                               void* y, void* q, float* scale, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int format = !q ? kNoQ : q_dtype == MOE_I8 ? kInt8 : kE4M3;
  return dtype == MOE_BF16
             ? norm<true>(format, x, residual, weight, eps, T, H, total, y, q, scale, s)
             : norm<false>(format, x, residual, weight, eps, T, H, total, y, q, scale, s);
}

hipError_t launch_quantize_int8(const void* x, int dtype, int64_t rows, int cols, void* q,
                                float* scale, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  return dtype == MOE_BF16 ? rows_to_int8<true>(x, (uint32_t)rows, cols, q, scale, s)
                           : rows_to_int8<false>(x, (uint32_t)rows, cols, q, scale, s);
}

}  // namespace moe
