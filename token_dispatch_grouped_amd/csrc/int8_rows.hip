// Quantisation to 8-bit integers for the experts' products: activation rows with
// one scale per row (dynamic, taken from the row itself), weights with one scale
// per output channel (once, before serving).
//
//   scale = max(max|a| / 127, 2^-126),  q = rint(a * (1 / scale))
//
// so a = q * scale to within half a step, a row of zeros gives q = 0, and no
// division by zero or overflow of 1 / scale can occur. A row (or channel) that
// holds an infinity or a NaN gets scale = NaN and q = 0: every product with it is
// NaN, as it would be in floating point.
//
// Both operands of the products are kept in K-blocks of 64: block kb of a matrix
// of R rows holds [R][64] bytes, columns 64 kb .. 64 kb + 63 of every row, zero
// past the last column. A K = 64 stage of a tile is then one contiguous run.
// Everything here is bound by HBM: a row is read once and its codes written once.
#include <math.h>

#include "int8_code.h"
#include "int8_plan.h"

namespace moe {
namespace {

using namespace rows;
using namespace int8;

template <int G>
constexpr int block_threads() { return G > 256 ? G : 256; }

// Rows [0, N_loc) of the local segment: row r is row perm[seg0 + r] / k of src
// (perm != nullptr: the dispatch's row gather) or row r. G threads per row, VPT
// vectors of 8 bf16 per thread; the row's K-blocks are filled up with zeros. With
// `plan`, one more workgroup (the first) lists the tiles of the call's GEMM launches.
template <int G, int VPT>
__global__ __launch_bounds__(block_threads<G>()) void quantize_rows_kernel(
    const uint4* __restrict__ src, const int32_t* __restrict__ perm, const int32_t* __restrict__ offsets,
    uint8_t* __restrict__ q, float* __restrict__ scale, int e_begin, int e_end, int k, int64_t T, int cols_vec,
    int kblocks, int64_t n_max, void* __restrict__ plan, int tile_rows) {
  constexpr int kRows = block_threads<G>() / G;
  __shared__ uint32_t lds[2][G > kWave ? G / kWave : 1];
  int turn = 0;
  const int planners = plan != nullptr ? 1 : 0;
  if (static_cast<int>(blockIdx.x) < planners) {
    int* count = static_cast<int*>(plan);
    int8::RowGroup* groups = reinterpret_cast<int8::RowGroup*>(static_cast<char*>(plan) + int8::kPlanHeader);
    const int e_loc = e_end - e_begin, n = static_cast<int>(n_max);
    if (tile_rows == kTallRows) plan_tiles<kTallRows, kTallMerge>(offsets, e_begin, e_loc, n, count, groups);
    else if (tile_rows == kShortRows) plan_tiles<kShortRows, 0>(offsets, e_begin, e_loc, n, count, groups);
    else plan_tiles<kThinRows, 0>(offsets, e_begin, e_loc, n, count, groups);
    return;
  }
  const int64_t block = static_cast<int64_t>(blockIdx.x) - planners;
  const int64_t blocks = static_cast<int64_t>(gridDim.x) - planners;
  const int seg0 = offsets[e_begin];
  const int64_t n_loc = min(static_cast<int64_t>(offsets[e_end] - seg0), n_max);
  const int li = static_cast<int>(threadIdx.x) % G;
  for (int64_t r0 = block * kRows; r0 < n_loc; r0 += blocks * kRows) {
    const int64_t r = r0 + threadIdx.x / G;
    const bool live = r < n_loc;
    const int64_t from = !live ? 0 : perm != nullptr ? perm[seg0 + r] / k : r;
    const int n = live && (perm == nullptr || (from >= 0 && from < T)) ? cols_vec : 0;
    uint4 v[VPT];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * G + li;
      v[i] = c < n ? src[from * cols_vec + c] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) top = Max::apply(top, amax8(v[i]));
    top = group_reduce<G, Max>(top, lds[turn]);
    turn ^= 1;
    float sc, inv;
    scale_of(top, &sc, &inv);
    if (live && li == 0) scale[r] = sc;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * G + li;
      if (live && c < kblocks * 8) {
        float f[8];
        Vec16<true>::unpack(v[i], f);
        *reinterpret_cast<uint2*>(q + (static_cast<int64_t>(c >> 3) * n_max + r) * 64 + (c & 7) * 8) = codes8(f, inv);
      }
    }
  }
}

// Weights [K, N] of each expert (row-major, N-contiguous) to codes in K-blocks
// [K / 64][N][64] with one scale per channel. A workgroup takes 64 channels of an
// expert: a pass for the channels' largest values, then a pass that turns 64 x 64
// blocks through LDS.
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_weights_kernel(const void* __restrict__ w, uint8_t* __restrict__ q,
                                                               float* __restrict__ scale, int K, int N) {
  __shared__ uint32_t tops[4][64];
  __shared__ float invs[64];
  __shared__ uint32_t turn[64][17];  // [channel][16 words of 4 codes + 1]
  const int tiles = (N + 63) / 64;
  const int64_t e = blockIdx.x / tiles;
  const int n0 = static_cast<int>(blockIdx.x % tiles) * 64;
  const int lane = lane_id(), wv = static_cast<int>(threadIdx.x) / kWave;
  const int n = n0 + lane;
  auto at = [&](int k) -> float {
    const int64_t i = (e * K + k) * N + n;
    return BF16 ? bf16_to_f32(static_cast<const uint16_t*>(w)[i]) : static_cast<const float*>(w)[i];
  };
  uint32_t top = 0;
  if (n < N)
#pragma unroll 8
    for (int k = wv; k < K; k += 4) top = Max::apply(top, abs_bits(at(k)));
  tops[wv][lane] = top;
  __syncthreads();
  if (wv == 0) {
    for (int i = 1; i < 4; ++i) top = Max::apply(top, tops[i][lane]);
    float sc, inv;
    scale_of(top, &sc, &inv);
    invs[lane] = inv;
    if (n < N) scale[e * N + n] = sc;
  }
  __syncthreads();
  const float inv = invs[lane];
  const int kblocks = (K + 63) / 64;
  for (int kb = 0; kb < kblocks; ++kb) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int kw = wv * 4 + j;  // word kw: rows 64 kb + 4 kw ..
      uint32_t word = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int k = kb * 64 + kw * 4 + b;
        if (n < N && k < K) word |= code(at(k), inv) << (8 * b);
      }
      turn[lane][kw] = word;
    }
    __syncthreads();
    uint32_t* out = reinterpret_cast<uint32_t*>(q) + ((e * kblocks + kb) * static_cast<int64_t>(N) + n0) * 16;
    for (int i = threadIdx.x; i < 64 * 16; i += 256)
      if (n0 + i / 16 < N) out[i] = turn[i / 16][i % 16];
    __syncthreads();
  }
}

template <int G, int VPT>
hipError_t launch_rows(const void* src, const int32_t* perm, const int32_t* offsets, void* q, float* scale, int e_begin,
                       int e_end, int k, int64_t T, int cols, int64_t n_max, void* plan, int tile_rows, hipStream_t stream) {
  constexpr int kRows = block_threads<G>() / G;
  // n_max may be many times the local rows: workgroups take turns, eight per CU
  const int64_t blocks = (n_max + kRows - 1) / kRows;
  hipLaunchKernelGGL((quantize_rows_kernel<G, VPT>), dim3(static_cast<unsigned>(blocks < 2048 ? blocks : 2048) + (plan != nullptr ? 1u : 0u)),
                     dim3(block_threads<G>()), 0, stream, static_cast<const uint4*>(src), perm, offsets,
                     static_cast<uint8_t*>(q), scale, e_begin, e_end, k, T, cols / 8, (cols + 63) / 64, n_max, plan,
                     tile_rows);
  return hipGetLastError();
}

}  // namespace

int int8_kblocks(int K) { return (K + 63) / 64; }

int64_t int8_max_k() { return 65536; }

// Which workgroups a call's products use, from the rows per expert that uniform routing gives
// (the real counts are on the device only; any choice is right for any counts): the one whose
// launches would take the least time, in microseconds, by what single launches measured. A launch
// takes no less than its weights at 6.6 TB/s.
//
// few    3 + the longer of 0.06 (wide: 0.1) per K-block, as a wave's loads wait for each other over a
//        quarter of K, and the bytes of all workgroups, 2 or 4 KB per K-block each, at 8.5 TB/s (mostly
//        L2), 1.5 for each time they fill the chip (three a CU), and 1.3 times as often what a
//        workgroup takes to quantise its rows: 0.6 + 0.25 per 1024 of K for each row (waves: four rows)
// thin   6 (with the quantising launch), 0.12 per K-block, 6 KB per K-block, else as few
// short  7 + 0.4 per K stage while each tile has a CU to itself; past that 6 + rounds of two tiles
//        per CU, 1.05 per stage + 0.8 (its products, and 1.5 times tall's bytes through LDS)
// tall   4 + rounds of one tile per CU, 0.8 per stage + 14 (the fill, and the epilogue that nothing
//        overlaps)
// A round that is at most half full costs 0.55 (tall: its tiles are halved). Whole calls (graph
// replays): one token, 8 experts of 1512 x 824: few 10 us, thin 16; 14 tokens x 2 of 4, 1 here, 944 x
// 1928: few 13, thin 18; 347 x 4 of 64, 1176 x 344: few 56, thin 35, short 30; 8 experts, 64 tokens x 2,
// 1024 x 3584: thin 34, short 42; 8 experts of 1024 rows, 4096 x 4096: short 458, tall 486; 4096 x
// 14336 (16384 tokens): short 2905, tall 2718; 16 experts of 256 rows, 2880 x 2880: short 177, tall 164.
int int8_tile_rows(int64_t T, int k, int E, int e_loc, int d, int d_ff) {
  const double rows = static_cast<double>(T) * k / E;  // per expert
  const double experts = fmax(1.0, e_loc * -expm1(-rows));  // that have any
  const double per = fmax(rows * e_loc / experts, 1.0);
  const double cus = device_cu_count();
  auto rounds = [](double r) {
    const double whole = floor(r), part = r - whole;
    return whole + (whole > 0 && part < 0.02 ? 0.0 : part <= 0.5 ? 0.55 : 1.0);
  };
  const double few_tiles = experts * ceil(per / kFewRows);
  const double thin_tiles = experts * ceil(per / kThinRows);
  const double short_tiles = experts * ceil(per / kShortRows);
  // in rounds, a light last tile counts half; counts that scatter leave light tiles more than their mean
  const double s_rest = fmod(per, kShortRows), t_rest = fmod(per, kTallRows);
  const double short_cost =
      experts * (floor(per / kShortRows) + (s_rest > 64 ? 1.0 : s_rest > 0 ? 0.5 : 0.0) + (per >= 64 ? 0.2 : 0.0));
  const double tall_cost =
      experts * fmax(1.0, floor(per / kTallRows) + (t_rest > 128 ? 1.0 : t_rest > kTallMerge ? 0.5 : 0.0));
  const double tall_more = per > 512 ? fmin(0.3, 0.04 * experts) : 0.0;
  double few = 0, thin = 0, shorter = 0, tall = 0;
  for (int i = 0; i < 2; ++i) {
    const int K = i ? d_ff : d, N = i ? d : d_ff;
    const double st = int8_kblocks(K), cols = (N + (i ? 255 : 127)) / (i ? 256 : 128);
    const double least = experts * K * N * (i ? 1.0 : 2.0) / 6.6e6;
    const int few_cols = int8_few_columns(T, k, e_loc, N, i == 0);
    const double few_groups = few_tiles * ((N + few_cols - 1) / few_cols), fills = few_groups / (3 * cus);
    const double quantized = fmin(per, kFewRows);  // rows of a workgroup
    const double turns = int8_few_waves(T, k, E, K) ? ceil(quantized / 4) : quantized;
    const double block = few_cols * (i ? 64 : 128);  // bytes of a workgroup's K-block
    few += 3 + fmax(fmax((block > 2048 ? 0.1 : 0.06) * st, few_groups * st * block / 8.5e6) + 1.5 * fills +
                        fmax(1.0, 1.3 * fills) * turns * (0.6 + K / 4096.0), least);
    const double thin_groups = thin_tiles * ((N + (i ? 63 : 31)) / (i ? 64 : 32));
    thin += 6 + fmax(fmax(0.12 * st, thin_groups * st * 6e3 / 8.5e6) + 1.5 * thin_groups / (3 * cus), least);
    const double s = short_cost * cols / (2 * cus);
    shorter += short_tiles * cols <= cus ? 7 + fmax(0.4 * st, least) : 6 + fmax(rounds(s) * (1.05 * st + 0.8), least);
    tall += 4 + fmax((rounds(tall_cost * cols / cus) + tall_more) * 0.8 * (st + 18), least);
  }
  if (few <= fmin(thin, fmin(shorter, tall)) && rows <= 64 && int8_few_fits(T, d > d_ff ? d : d_ff)) return kFewRows;
  // a thin launch's grid holds every tile there could be: a share that might get far more rows takes another
  const int64_t n_max = T * (k < e_loc ? k : e_loc);
  if (thin <= fmin(shorter, tall) && max_row_tiles(n_max, e_loc, kThinRows) <= kThinTiles) return kThinRows;
  return tall <= shorter ? kTallRows : kShortRows;
}

// Room for the list of any choice.
size_t int8_plan_bytes(int64_t n_max, int e_loc) {
  return kPlanHeader + static_cast<size_t>(max_row_tiles(n_max, e_loc, kThinRows)) * sizeof(RowGroup);
}

hipError_t launch_quantize_rows(const void* src, const int32_t* perm, const int32_t* offsets, void* q, float* scale,
                                int e_begin, int e_end, int k, int64_t T, int cols, int64_t n_max, void* plan,
                                int tile_rows, hipStream_t stream) {
  const int vec = int8_kblocks(cols) * 8;  // the padded row, in vectors of 8 elements
#define MOE_QROWS(G, VPT) \
  return launch_rows<G, VPT>(src, perm, offsets, q, scale, e_begin, e_end, k, T, cols, n_max, plan, tile_rows, stream)
  if (vec <= 64) MOE_QROWS(64, 1);
  if (vec <= 256) MOE_QROWS(64, 4);
  if (vec <= 512) MOE_QROWS(64, 8);
  if (vec <= 1024) MOE_QROWS(256, 4);
  if (vec <= 2048) MOE_QROWS(256, 8);
  if (vec <= 4096) MOE_QROWS(1024, 4);
  MOE_QROWS(1024, 8);
#undef MOE_QROWS
}

hipError_t launch_quantize_weights(const void* w, void* q, float* scale, int e_loc, int K, int N, bool bf16,
                                   hipStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(e_loc) * static_cast<unsigned>((N + 63) / 64);
  if (bf16)
    hipLaunchKernelGGL(quantize_weights_kernel<true>, dim3(blocks), dim3(256), 0, stream, w, static_cast<uint8_t*>(q),
                       scale, K, N);
  else
    hipLaunchKernelGGL(quantize_weights_kernel<false>, dim3(blocks), dim3(256), 0, stream, w, static_cast<uint8_t*>(q),
                       scale, K, N);
  return hipGetLastError();
}

}  // namespace moe
