// quant.hip -- 8-bit block quantisation of rows and of weights, and the
// dispatch copy that quantises token rows on their way into the send buffer
// (the permute copy of the explainer's section 3 item 5 with a payload of one
// byte an element, so the exchange carries half of bf16's bytes). The scales
// and their rounding are those of quant.h.
//
// Bound by HBM bytes: each element is read once and written once (k times by
// the dispatch copy) as one byte, each scale is 4 bytes per 128 elements.
#include <type_traits>

#include "device.h"
#include "launch.h"
#include "quant.h"

namespace moe {
namespace {

constexpr int kBlock = 256;

// Streaming store of a lane's e4m3 bytes.
__device__ __forceinline__ void store_q(void* p, uint2 v) {
  typedef uint32_t v2u __attribute__((ext_vector_type(2)));
  __builtin_nontemporal_store(v2u{v.x, v.y}, static_cast<v2u*>(p));
}
__device__ __forceinline__ void store_q(void* p, uint32_t v) {
  __builtin_nontemporal_store(v, static_cast<uint32_t*>(p));
}

// Rows: QuantVec::kLanes consecutive lanes hold one group of 128 columns. Flat over
// (row, group, lane of the group); the last group of a row may be short (cols %
// 128, a multiple of 16). nvec: 16-byte vectors of a row. 128 x 4096 bf16: 2.5 us,
// launch latency.
template <bool kBF16>
__global__ __launch_bounds__(kBlock) void quantize_rows_kernel(const v4u* __restrict__ x,
                                                               uint32_t total, uint32_t groups,
                                                               uint32_t nvec, uint8_t* __restrict__ q,
                                                               float* __restrict__ scale) {
  typedef QuantVec<kBF16> Vec;
  const uint32_t i = blockIdx.x * (uint32_t)kBlock + threadIdx.x;
  const uint32_t grp = i / Vec::kLanes;  // group of the whole array: row * groups + group
  const uint32_t row = grp / groups;
  const uint32_t col = (grp - row * groups) * Vec::kLanes + i % Vec::kLanes;
  const bool ok = i < total && col < nvec;
  const size_t at = (size_t)row * nvec + col;
  Vec v = {v4u{0, 0, 0, 0}};
  if (ok) v.v = load_stream(x + at);
  const int p = scale_exponent(lanes_max<Vec::kLanes>(v.amax()));
  if (ok) store_q(q + at * Vec::N, v.quantize(power_of_two(-p)));
  if (i < total && i % Vec::kLanes == 0) scale[grp] = power_of_two(p);
}

// Blocks of 128 x 128: one thread block each, its elements held in registers
// between the maximum and the rounding, so x is read once. One 16-byte vector a
// lane and row: 16 x 2816 x 4096 bf16 in 93 us, 5.9 TB/s (two vectors, half the
// loads in flight: 105 us).
template <bool kBF16>
__global__ __launch_bounds__(kBlock) void quantize_blocks_kernel(
    const v4u* __restrict__ x, uint32_t rows, uint32_t rblocks, uint32_t cblocks, uint32_t nvec,
    uint8_t* __restrict__ q, float* __restrict__ scale) {
  typedef QuantVec<kBF16> Vec;
  constexpr int kPer = kBlock / Vec::kLanes;    // rows a pass
  constexpr int kPass = kQuantBlock / kPer;     // rows a thread holds
  __shared__ uint32_t part[kBlock / kWave];
  const uint32_t b = blockIdx.x;  // (batch, row block, column block)
  const uint32_t rb = b / cblocks, cb = b - rb * cblocks;
  const uint32_t batch = rb / rblocks, r0 = (rb - batch * rblocks) * kQuantBlock;
  const uint32_t col = cb * Vec::kLanes + threadIdx.x % Vec::kLanes;
  const uint32_t lr = threadIdx.x / Vec::kLanes;
  Vec v[kPass];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kPass; ++j) {
    const uint32_t r = r0 + lr + j * kPer;
    v[j].v = v4u{0, 0, 0, 0};
    if (col < nvec && r < rows) v[j].v = load_stream(x + ((size_t)batch * rows + r) * nvec + col);
  }
#pragma unroll
  for (int j = 0; j < kPass; ++j) {
    const uint32_t a = v[j].amax();
    m = a > m ? a : m;
  }
  m = lanes_max<kWave>(m);
  if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kBlock / kWave; ++w) m = part[w] > m ? part[w] : m;
  const int p = scale_exponent(m);
  const float inv = power_of_two(-p);
#pragma unroll
  for (int j = 0; j < kPass; ++j) {
    const uint32_t r = r0 + lr + j * kPer;
    if (col < nvec && r < rows)
      store_q(q + (((size_t)batch * rows + r) * nvec + col) * Vec::N, v[j].quantize(inv));
  }
  if (threadIdx.x == 0) scale[b] = power_of_two(p);
}

// Dispatch: the lane layout of quantize_rows_kernel over x [T][H]; each lane
// stores its bytes to the token's k send rows (picks without a row inside
// [0, nrows) are skipped), the group's first lane the scale. Bound by the
// scattered writes: 131072 rows of 7168 from 16384 tokens, 1.2 GB in 222 us, 5.4
// TB/s; 24576 rows of 2048 in 14 us.
template <bool kBF16, int KMAX>
__global__ __launch_bounds__(kBlock) void dispatch_fp8_kernel(
    const v4u* __restrict__ x, const int32_t* __restrict__ pos, int k, uint32_t total,
    uint32_t groups, uint32_t nvec, uint32_t nrows, uint8_t* __restrict__ q,
    float* __restrict__ scale) {
  typedef QuantVec<kBF16> Vec;
  const uint32_t i = blockIdx.x * (uint32_t)kBlock + threadIdx.x;
  const uint32_t grp = i / Vec::kLanes;
  const uint32_t t = grp / groups, g = grp - t * groups;
  const uint32_t col = g * Vec::kLanes + i % Vec::kLanes;
  const bool live = i < total;
  const bool ok = live && col < nvec;
  Vec v = {v4u{0, 0, 0, 0}};
  if (ok) v.v = load_stream(x + (size_t)t * nvec + col);
  int32_t P[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) P[j] = (live && j < k) ? pos[(size_t)t * k + j] : -1;
  const int p = scale_exponent(lanes_max<Vec::kLanes>(v.amax()));
  const typename Vec::Out out = v.quantize(power_of_two(-p));
  const float s = power_of_two(p);
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    if ((uint32_t)P[j] < nrows) {
      if (ok) store_q(q + ((size_t)P[j] * nvec + col) * Vec::N, out);
      if (i % Vec::kLanes == 0) scale[(size_t)P[j] * groups + g] = s;
    }
  }
}

}  // namespace

hipError_t launch_quantize(const void* x, int dtype, int64_t batch, int64_t rows, int cols,
                           int block_rows, void* q, float* scale, hipStream_t s) {
  if (batch == 0 || rows == 0) return hipSuccess;
  const int per_vec = dtype == MOE_BF16 ? 8 : 4;  // elements of a 16-byte vector
  const uint32_t nvec = (uint32_t)(cols / per_vec);
  const uint32_t groups = (uint32_t)((cols + kQuantBlock - 1) / kQuantBlock);
  const v4u* xv = static_cast<const v4u*>(x);
  uint8_t* qv = static_cast<uint8_t*>(q);
  if (block_rows == 1) {
    const uint32_t total = (uint32_t)(batch * rows * groups * (kQuantBlock / per_vec));
    const dim3 grid((total + kBlock - 1) / kBlock);
    return dtype == MOE_BF16 ? launch(quantize_rows_kernel<true>, grid, dim3(kBlock), 0, s, xv,
                                      total, groups, nvec, qv, scale)
                             : launch(quantize_rows_kernel<false>, grid, dim3(kBlock), 0, s, xv,
                                      total, groups, nvec, qv, scale);
  }
  const uint32_t rblocks = (uint32_t)((rows + kQuantBlock - 1) / kQuantBlock);
  const dim3 grid((unsigned)(batch * rblocks * groups));
  return dtype == MOE_BF16 ? launch(quantize_blocks_kernel<true>, grid, dim3(kBlock), 0, s, xv,
                                    (uint32_t)rows, rblocks, groups, nvec, qv, scale)
                           : launch(quantize_blocks_kernel<false>, grid, dim3(kBlock), 0, s, xv,
                                    (uint32_t)rows, rblocks, groups, nvec, qv, scale);
}

hipError_t launch_dispatch_fp8(const void* x, int dtype, const int32_t* pos, int T, int k, int H,
                               int64_t send_rows, void* send_q, float* send_scale, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int per_vec = dtype == MOE_BF16 ? 8 : 4;
  const uint32_t nvec = (uint32_t)(H / per_vec);
  const uint32_t groups = (uint32_t)((H + kQuantBlock - 1) / kQuantBlock);
  const uint32_t total = (uint32_t)T * groups * (kQuantBlock / per_vec);
  const dim3 grid((total + kBlock - 1) / kBlock);
  auto go = [&](auto kmax) {
    constexpr int KM = decltype(kmax)::value;
    auto run = [&](auto kernel) {
      return launch(kernel, grid, dim3(kBlock), 0, s, static_cast<const v4u*>(x), pos, k, total,
                    groups, nvec, (uint32_t)send_rows, static_cast<uint8_t*>(send_q), send_scale);
    };
    return dtype == MOE_BF16 ? run(dispatch_fp8_kernel<true, KM>)
                             : run(dispatch_fp8_kernel<false, KM>);
  };
  if (k <= 2) return go(std::integral_constant<int, 2>{});
  if (k <= 8) return go(std::integral_constant<int, 8>{});
  return go(std::integral_constant<int, 32>{});
}

}  // namespace moe
