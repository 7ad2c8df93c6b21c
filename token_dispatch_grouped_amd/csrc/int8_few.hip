// The experts' FFN in 8-bit integers for a few rows per expert (decoding): two launches,
// each quantising its own rows.
//
//   gate/up: rows of x (through perm) -> codes in LDS; H = silu(G) * U (bf16)
//   down:    rows of H -> codes in LDS; Y (bf16)
//
// With a handful of rows the weights are streamed once for almost no arithmetic, so
// what counts is bytes in flight and launches. A workgroup takes up to 16 rows of an
// expert and 16 * FRAGS weight channels over all of K; its four waves take a quarter of
// K each and ask for their weights, straight into registers, before anything else.
// While those are on their way the workgroup quantises its rows (each workgroup of an
// expert does so again: a few KB from L2 next to its 100 KB of weights). 32 tokens x 4 of
// 128 experts of 2880 x 2880: 306 us, 2.0 GB of weights at 6.6 TB/s; one token of 4 of 32
// experts of 1000 x 1480: 6.0 + 4.8 us for 18 MB, bound by its chains of loads (offsets, row
// ids, rows, then the product).
// v_mfma_i32_16x16x64_i8: 16 channels x 64 K values of the K-blocked weights are one
// contiguous KB, lane L's 16 bytes at (L & 15) * 64 + (L >> 4) * 16. Integer sums are
// exact, so the quarters of K are joined in any order with the same bits.
#include "int8_code.h"
#include "int8_plan.h"

namespace moe {
namespace {

using namespace int8;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kFewTokens = 128;  // of a call at most
constexpr int kHeld = 4;    // vectors of a row a thread holds between its two passes
constexpr int kMaxCodes = 48 * 1024 - 128;  // with the sums 64 KB, and two workgroups a CU at least

typedef int i32x4 __attribute__((ext_vector_type(4)));

// rows of a workgroup's turn
__host__ __device__ constexpr int few_rows(int64_t T) { return T < kFewRows ? static_cast<int>(T) : kFewRows; }
__host__ __device__ constexpr int code_stride(int kblocks) { return kblocks * 64 + 16; }  // rows fall into different banks

// FRAGS 16-channel blocks of a workgroup (SwiGLU: half gate, half up), AHEAD K-blocks that
// a wave has in flight.
template <bool SWIGLU, int FRAGS, int AHEAD>
struct Weights {
  static constexpr int NO = SWIGLU ? FRAGS / 2 : FRAGS;  // blocks of output columns
  const uint8_t* base;  // the expert's
  int64_t block_bytes;  // of one K-block
  int lo, hi;           // this wave's K-blocks, a quarter of all
  uint32_t off[FRAGS];
  i32x4 b[AHEAD][FRAGS];
  float scale[FRAGS];   // of this lane's channels, for the end

  __device__ Weights(const uint8_t* w, int e, int n0, int kblocks, int N) {
    const int lane = lane_id(), wv = uniform(static_cast<int>(threadIdx.x) / kWave);
    const int64_t channels = SWIGLU ? 2 * static_cast<int64_t>(N) : N;
    block_bytes = channels * 64;
    base = w + e * block_bytes * kblocks;
    lo = kblocks * wv / kWaves;
    hi = kblocks * (wv + 1) / kWaves;
#pragma unroll
    for (int f = 0; f < FRAGS; ++f) {
      const int col = min(n0 + 16 * (f % NO) + (lane & 15), N - 1);  // channels past N are read again and not stored
      off[f] = static_cast<uint32_t>(col + (f >= NO ? N : 0)) * 64u + static_cast<uint32_t>(lane >> 4) * 16u;
    }
  }
  __device__ void load_scales(const float* __restrict__ w_scale, int e) {
#pragma unroll
    for (int f = 0; f < FRAGS; ++f) scale[f] = w_scale[e * (block_bytes / 64) + off[f] / 64];
  }
  __device__ void load(int kb0) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (kb0 + u < hi) {
        const uint8_t* p = base + (kb0 + u) * block_bytes;
#pragma unroll
        for (int f = 0; f < FRAGS; ++f) b[u][f] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(p + off[f]));
      }
  }
};

// The four quarters of K joined, scaled and stored: `rows` rows from row r0 of `out`.
// part: [wave][RT * FRAGS][lane], lane l's element j of a block is row (l >> 4) * 4 + j,
// channel l & 15; a thread takes one element of every block.
template <bool SWIGLU, int FRAGS, int RT>
__device__ __forceinline__ void finish(const i32x4* part, const float* row_scale, const float* w_scale,
                                       __bf16* __restrict__ out, int64_t r0, int rows, int n0, int N) {
  constexpr int NO = SWIGLU ? FRAGS / 2 : FRAGS;
  const int lane = lane_id(), j = static_cast<int>(threadIdx.x) / kWave;
  auto sum = [&](int t, int f) {
    int s = 0;
#pragma unroll
    for (int q = 0; q < kWaves; ++q)
      s += reinterpret_cast<const int*>(part)[(((q * RT + t) * FRAGS + f) * kWave + lane) * 4 + j];
    return static_cast<float>(s);
  };
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = t * 16 + (lane >> 4) * 4 + j;
    if (row >= rows) continue;
    const float sa = row_scale[row];
#pragma unroll
    for (int f = 0; f < NO; ++f) {
      const int col = n0 + 16 * f + (lane & 15);
      if (col < N) {
        float v = sum(t, f) * w_scale[f] * sa;
        if constexpr (SWIGLU) v = gemm::silu_fast(v) * (sum(t, f + NO) * w_scale[f + NO] * sa);
        out[(r0 + row) * N + col] = static_cast<__bf16>(v);
      }
    }
  }
}

// The workgroup quantises its rows, G threads a row, or (CODES) finds them in 8 bits already: src
// then holds codes [kblocks][T][64], src_scale their scales (32 tokens x 4 of 128 experts of 2880 x 2880: 272.6 us
// instead of 277.2). Three waves per SIMD.
template <bool SWIGLU, int FRAGS, int AHEAD, int G, bool CODES>
__global__ __launch_bounds__(kThreads, 3) void int8_few_kernel(
    const uint4* __restrict__ src, const float* __restrict__ src_scale, const int32_t* __restrict__ perm, const int32_t* __restrict__ offsets,
    const uint8_t* __restrict__ w, const float* __restrict__ w_scale, __bf16* __restrict__ out, int e_begin, int k,
    int64_t T, int cols_vec, int kblocks, int N, int64_t n_max) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ i32x4 part[kWaves * FRAGS * kWave];
  __shared__ float scales[kFewRows];
  __shared__ uint32_t tops[2][kWaves];
  using Wt = Weights<SWIGLU, FRAGS, AHEAD>;
  const int tid = threadIdx.x, lane = lane_id(), wv = uniform(tid / kWave);
  const int e = blockIdx.y;
  const int seg0 = offsets[e_begin];
  const int start = static_cast<int>(min(static_cast<int64_t>(offsets[e_begin + e] - seg0), n_max));
  const int end = static_cast<int>(min(static_cast<int64_t>(offsets[e_begin + e + 1] - seg0), n_max));
  // one turn for most experts; their number has no bound but n_max, as topk_idx may repeat an id in a token
  const int tile = few_rows(T);
  int r0 = start + static_cast<int>(blockIdx.z) * tile;
  if (r0 >= end) return;
#pragma clang loop unroll(disable)
  for (;;) {
    // vmcnt(0), at once in the first turn: without it the compiler has every weight load wait, in the first
    // turn too, for a load of the turn before that might still write its registers (one token: 2.4 us)
    __builtin_amdgcn_s_waitcnt(0x0F70);
    const int R = min(tile, end - r0);
    const int n0 = static_cast<int>(blockIdx.x) * 16 * Wt::NO;
    Wt wt(w, e, n0, kblocks, N);
    wt.load(wt.lo);
    wt.load_scales(w_scale, e);
    __builtin_amdgcn_sched_barrier(0);  // in flight before anything else

    // the rows' codes
    const int stride = code_stride(kblocks);
    const int li = tid % G;
    for (int r = G == kThreads ? 0 : wv; r < R; r += kThreads / G) {
      int64_t from = r0 + r;
      if (perm != nullptr) from = perm[seg0 + r0 + r] / k;
      const int n = perm == nullptr || (from >= 0 && from < T) ? cols_vec : 0;
      if constexpr (CODES) {
        if (li == 0) scales[r] = n != 0 ? src_scale[from] : kMinScale;
        for (int c = li; c < kblocks * 4; c += G)
          *reinterpret_cast<uint4*>(smem + r * stride + c * 16) =
              n != 0 ? src[((c >> 2) * T + from) * 4 + (c & 3)] : make_uint4(0, 0, 0, 0);
        continue;
      }
      const uint4* row = src + from * cols_vec;
      uint4 v[kHeld];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int c = i * G + li;
        v[i] = c < n ? row[c] : make_uint4(0, 0, 0, 0);
      }
      for (int c = kHeld * G + li; c < n; c += G) top = rows::Max::apply(top, amax8(row[c]));
#pragma unroll
      for (int i = 0; i < kHeld; ++i) top = rows::Max::apply(top, amax8(v[i]));
      top = rows::group_reduce<G, rows::Max>(top, tops[r & 1]);
      float sc, inv;
      scale_of(top, &sc, &inv);
      if (li == 0) scales[r] = sc;
      char* codes = smem + r * stride;
      auto put = [&](int c, const uint4& a) {
        float f[8];
        rows::Vec16<true>::unpack(a, f);
        *reinterpret_cast<uint2*>(codes + c * 8) = codes8(f, inv);
      };
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int c = i * G + li;
        if (c < kblocks * 8) put(c, v[i]);  // zeros past the last column
      }
      for (int c = kHeld * G + li; c < kblocks * 8; c += G) put(c, c < n ? row[c] : make_uint4(0, 0, 0, 0));
    }
    __syncthreads();

    // lanes of rows past the last read the last row's codes; their sums are not stored
    const char* mine = smem + min(lane & 15, R - 1) * stride + (lane >> 4) * 16;
    i32x4 acc[FRAGS];
#pragma unroll
    for (int f = 0; f < FRAGS; ++f) acc[f] = i32x4{0, 0, 0, 0};
    for (int kb0 = wt.lo; kb0 < wt.hi; kb0 += AHEAD) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if (kb0 + u < wt.hi) {
          const i32x4 a = *reinterpret_cast<const i32x4*>(mine + (kb0 + u) * 64);
#pragma unroll
          for (int f = 0; f < FRAGS; ++f)
            acc[f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, wt.b[u][f], acc[f], 0, 0, 0);
        }
      if (kb0 + AHEAD < wt.hi) wt.load(kb0 + AHEAD);
    }
#pragma unroll
    for (int f = 0; f < FRAGS; ++f) part[(wv * FRAGS + f) * kWave + lane] = acc[f];
    __syncthreads();
    finish<SWIGLU, FRAGS, 1>(part, scales, wt.scale, out, r0, R, n0, N);
    r0 += static_cast<int>(gridDim.z) * tile;
    if (r0 >= end) break;
    __syncthreads();  // the next turn writes the codes, scales and sums again
  }
}

// Up to 32 rows of an expert whose codes are there already: as above, the rows' codes
// loaded like the weights (a K-block of 16 rows is one contiguous KB as well).
template <bool SWIGLU, int FRAGS, int AHEAD>
__global__ __launch_bounds__(kThreads, 3) void int8_thin_kernel(
    const uint8_t* __restrict__ codes, const float* __restrict__ a_scale, const uint8_t* __restrict__ w,
    const float* __restrict__ w_scale, __bf16* __restrict__ out, const int* __restrict__ n_row_tiles,
    const RowGroup* __restrict__ groups, int kblocks, int N, int64_t n_max) {
  constexpr int RT = kThinRows / 16;
  __shared__ i32x4 part[kWaves * RT * FRAGS * kWave];
  __shared__ float scales[kThinRows];
  using Wt = Weights<SWIGLU, FRAGS, AHEAD>;
  const int tid = threadIdx.x, lane = lane_id(), wv = uniform(tid / kWave);
  // column blocks fastest
  const int cols = (N + 16 * Wt::NO - 1) / (16 * Wt::NO), q = static_cast<int>(blockIdx.x) / cols;
  const int n0 = (static_cast<int>(blockIdx.x) - q * cols) * 16 * Wt::NO;
  if (q >= *n_row_tiles) return;
  const RowGroup g = groups[q];
  const int r0 = g.row0 + g.index * kThinRows;
  const int R = min(kThinRows, g.row_end - r0);
  Wt wt(w, g.expert, n0, kblocks, N);
  uint32_t off[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
    off[t] = static_cast<uint32_t>(min(16 * t + (lane & 15), R - 1)) * 64u + static_cast<uint32_t>(lane >> 4) * 16u;
  const uint8_t* rows0 = codes + static_cast<int64_t>(r0) * 64;
  i32x4 a[AHEAD][RT];
  auto load = [&](int kb0) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (kb0 + u < wt.hi) {
        const uint8_t* p = rows0 + (kb0 + u) * n_max * 64;
#pragma unroll
        for (int t = 0; t < RT; ++t) a[u][t] = *reinterpret_cast<const i32x4*>(p + off[t]);
      }
    wt.load(kb0);
  };
  load(wt.lo);
  wt.load_scales(w_scale, g.expert);
  if (tid < R) scales[tid] = a_scale[r0 + tid];
  i32x4 acc[RT][FRAGS];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int f = 0; f < FRAGS; ++f) acc[t][f] = i32x4{0, 0, 0, 0};
  for (int kb0 = wt.lo; kb0 < wt.hi; kb0 += AHEAD) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (kb0 + u < wt.hi) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int f = 0; f < FRAGS; ++f)
            acc[t][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u][t], wt.b[u][f], acc[t][f], 0, 0, 0);
      }
    if (kb0 + AHEAD < wt.hi) load(kb0 + AHEAD);
  }
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int f = 0; f < FRAGS; ++f) part[((wv * RT + t) * FRAGS + f) * kWave + lane] = acc[t][f];
  __syncthreads();
  finish<SWIGLU, FRAGS, RT>(part, scales, wt.scale, out, r0, R, n0, N);
}

template <bool SWIGLU, int FRAGS, int AHEAD, int G, bool CODES = false>
hipError_t launch_one(const void* src, const float* src_scale, const int32_t* perm, const int32_t* offsets, const void* w,
                      const float* w_scale, void* out, int E, int e_begin, int e_loc, int k, int64_t T, int K, int N,
                      int64_t n_max, hipStream_t stream) {
  constexpr int cols = 16 * (SWIGLU ? FRAGS / 2 : FRAGS);
  const int kblocks = int8_kblocks(K);
  const int rows = few_rows(T);
  // Workgroups for twice the rows that uniform routing gives an expert, and no fewer than a quarter of what
  // one could get: an expert with more takes up to four turns, and few workgroups are empty (128 tokens,
  // 64 experts of 1024 x 1024: all on one expert 56 us in four turns, 96 in eight; spread 35 either way).
  const int64_t likely = min(max((2 * T * k + E - 1) / E, (T + 3) / 4), T);
  const dim3 grid(static_cast<unsigned>((N + cols - 1) / cols), static_cast<unsigned>(e_loc),
                  static_cast<unsigned>((likely + rows - 1) / rows));
  hipLaunchKernelGGL((int8_few_kernel<SWIGLU, FRAGS, AHEAD, G, CODES>), grid, dim3(kThreads),
                     static_cast<unsigned>(rows * code_stride(kblocks)), stream, static_cast<const uint4*>(src), src_scale, perm,
                     offsets, static_cast<const uint8_t*>(w), w_scale, static_cast<__bf16*>(out), e_begin, k, T, K / 8,
                     kblocks, N, n_max);
  return hipGetLastError();
}

template <bool SWIGLU>
hipError_t launch_product(const void* src, const float* src_scale, const int32_t* perm, const int32_t* offsets, const void* w,
                          const float* w_scale, void* out, int E, int e_begin, int e_loc, int k, int64_t T, int K,
                          int N, int64_t n_max, hipStream_t stream) {
  const bool narrow = int8_few_columns(T, k, e_loc, N, SWIGLU) == 16 * (SWIGLU ? 1 : 2);
#define MOE_FEW(F, A, G)                                                                                          \
  return launch_one<SWIGLU, F, A, G>(src, nullptr, perm, offsets, w, w_scale, out, E, e_begin, e_loc, k, T, K, N, n_max, \
                                     stream)
  if constexpr (SWIGLU) {  // h is bf16
    if (src_scale != nullptr) {
      if (narrow)
        return launch_one<true, 2, 6, kWave, true>(src, src_scale, perm, offsets, w, w_scale, out, E, e_begin, e_loc, k,
                                                   T, K, N, n_max, stream);
      return launch_one<true, 4, 4, kWave, true>(src, src_scale, perm, offsets, w, w_scale, out, E, e_begin, e_loc, k, T,
                                                 K, N, n_max, stream);
    }
  }
  if (int8_few_waves(T, k, E, K)) {
    if (narrow) MOE_FEW(2, 6, kWave);
    MOE_FEW(4, 4, kWave);
  }
  if (narrow) MOE_FEW(2, 6, kThreads);
  MOE_FEW(4, 4, kThreads);
#undef MOE_FEW
}

}  // namespace

// Output columns of a workgroup: narrow where wide ones would be fewer than four per CU (one token, 4 of
// 32 experts of 1000 x 1480: 11.2 us against 13.4; one token, 2 experts of 4096 x 14336: 59.6 against
// 63.5); the wide ones' longer runs stream better once they fill the chip (32 tokens, 128 experts
// of 2880 x 2880: 296 us against 342).
int int8_few_columns(int64_t T, int k, int e_loc, int N, bool swiglu) {
  const int wide = swiglu ? 32 : 64;
  const int64_t n_max = T * (k < e_loc ? k : e_loc), active = n_max < e_loc ? n_max : e_loc;
  return active * ((N + wide - 1) / wide) < 4 * device_cu_count() ? wide / 2 : wide;
}

// A wave quantises a row (four at a time) unless it is long, by how many there are: a wave holds 2048
// elements between its two passes and reads the others twice. 6 tokens x 3 of 8 experts, 520 x 640: 9.2
// us against 14.5 with all threads on one row after the other; one token of 64 experts, 608 x 10312:
// 32.4 against 26.2.
bool int8_few_waves(int64_t T, int k, int E, int K) {
  return K * static_cast<int64_t>(E) <= kHeld * kWave * 8 * max(T * k, static_cast<int64_t>(E));
}

// Whether the codes of a workgroup's rows fit its LDS; and not too many tokens, whatever their number per
// expert, as all of them may go to one (512 tokens, 64 experts of 1024 x 1024: all on one expert 70 us,
// thin 20; spread 49 both).
bool int8_few_fits(int64_t T, int K) {
  return T <= kFewTokens && few_rows(T) * code_stride(int8_kblocks(K)) <= kMaxCodes;
}

hipError_t launch_int8_few(const void* x, const float* x_scale, const int32_t* perm, const int32_t* offsets, const void* q_gu,
                           const float* s_gu, const void* q_dn, const float* s_dn, void* h, void* y, int d, int d_ff,
                           int E, int e_begin, int e_loc, int k, int64_t T, int64_t n_max, hipStream_t stream) {
  const hipError_t e =
      launch_product<true>(x, x_scale, perm, offsets, q_gu, s_gu, h, E, e_begin, e_loc, k, T, d, d_ff, n_max, stream);
  if (e != hipSuccess) return e;
  return launch_product<false>(h, nullptr, nullptr, offsets, q_dn, s_dn, y, E, e_begin, e_loc, k, T, d_ff, d, n_max, stream);
}

hipError_t launch_int8_thin(const void* a, const float* a_scale, const void* w, const float* w_scale, void* c,
                            const void* plan, int e_loc, int K, int N, int64_t n_max, bool swiglu, hipStream_t stream) {
  const int* count = static_cast<const int*>(plan);
  const int8::RowGroup* groups =
      reinterpret_cast<const int8::RowGroup*>(static_cast<const char*>(plan) + int8::kPlanHeader);
  const unsigned tiles = static_cast<unsigned>(int8::max_row_tiles(n_max, e_loc, int8::kThinRows));
  const int kblocks = int8_kblocks(K);
#define MOE_THIN(S, F, A)                                                                                         \
  hipLaunchKernelGGL((int8_thin_kernel<S, F, A>),                                                                 \
                     dim3(tiles * static_cast<unsigned>((N + 16 * (S ? F / 2 : F) - 1) / (16 * (S ? F / 2 : F)))), \
                     dim3(kThreads), 0, stream, static_cast<const uint8_t*>(a), a_scale,                          \
                     static_cast<const uint8_t*>(w), w_scale, static_cast<__bf16*>(c), count, groups, kblocks, N, \
                     n_max)
  if (swiglu) MOE_THIN(true, 4, 3);
  else MOE_THIN(false, 4, 3);
#undef MOE_THIN
  return hipGetLastError();
}

}  // namespace moe
