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
// (the real counts are on the device only; any choice is right for any counts):
//
// thin  (tiles of 32 rows) where the short tiles of a product are too few for the chip, as few
//       experts with few columns give. Graph replays: 8 experts, 64 tokens x 2, 1024 x 3584:
//       33.8 us against 41.6; 4 experts, 64 tokens, 4096 x 512: 22.6 against 34.2; but 32 experts,
//       64 tokens x 4, 1024 x 1024 (128 short tiles): 32.8 against 31.0, and 8 experts, 512 tokens x
//       2, 1024 x 3584 (128 rows each): 75 against 64. Its grid holds every tile there could be,
//       so a rank that might get far more rows than it will (a small share) takes the others.
// tall  where its rounds cost less than the short ones'. A round of tall tiles on 256 CUs
//       measured as its K stages + 18 (fill, and the epilogue that nothing overlaps), a round of short
//       tiles, two per CU, as 1.31 times its stages + 1 (1.5 times the bytes through LDS, but one tile
//       computes while the other waits); a round that is at most half full costs 0.55. 8 experts of 1024
//       rows: 4096 x 14336 tall 2718 us (16384 tokens), short 2905; 4096 x 4096 tall 486, short 458;
//       8 experts of 512 rows 4096 x 4096 tall 233, short 265; 16 of 256 rows 2880 x 2880 tall 164,
//       short 177; 16 of 1024 rows 1024 x 2048 tall 215, short 173.
// short otherwise.
int int8_tile_rows(int64_t T, int k, int E, int e_loc, int d, int d_ff) {
  const double rows = static_cast<double>(T) * k / E;  // per expert
  const double experts = rows * e_loc < 1.0 ? 1.0 : rows < 1.0 ? rows * e_loc : e_loc;
  const double cols[2] = {(d_ff + 127) / 128 * 1.0, (d + 255) / 256 * 1.0};
  const double stages[2] = {int8_kblocks(d) * 1.0, int8_kblocks(d_ff) * 1.0};
  const double cus = device_cu_count();
  const double short_tiles = experts * ceil(rows / kShortRows);
  const double fewest = fmin(short_tiles * cols[0], short_tiles * cols[1]);
  const double most = fmax(short_tiles * cols[0], short_tiles * cols[1]);
  const int64_t n_max = T * (k < e_loc ? k : e_loc);
  if (((fewest < cus / 4 && rows <= 64) || most < cus / 4) && max_row_tiles(n_max, e_loc, kThinRows) <= kThinTiles)
    return kThinRows;
  const double full = floor(rows / kTallRows), rest = rows - full * kTallRows;
  // a short last tile costs about half of a tall one; one of up to 32 rows rides along
  const double tall_tiles = experts * fmax(1.0, full + (rest > 128 ? 1.0 : rest > kTallMerge ? 0.5 : 0.0));
  auto rounds = [](double r) {
    const double whole = floor(r), part = r - whole;
    return whole + (part < 0.02 ? 0.0 : part <= 0.5 ? 0.55 : 1.0);
  };
  // counts that scatter around their mean leave a few tiles more than it says
  const double tall_more = experts > 1 && rows > 512 ? 0.3 : 0.0, short_more = 0.1;
  double tall = 0, shorter = 0;
  for (int i = 0; i < 2; ++i) {
    tall += (rounds(tall_tiles * cols[i] / cus) + tall_more) * (stages[i] + 18);
    shorter += (rounds(short_tiles * cols[i] / (2 * cus)) + short_more) * (1.31 * stages[i] + 1);
  }
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
