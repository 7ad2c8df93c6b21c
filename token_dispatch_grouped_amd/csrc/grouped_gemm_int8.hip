// Grouped expert GEMM in 8-bit integers: the experts' SwiGLU FFN on quantised rows
// and weights (int8_rows.hip), with exact int32 sums on the matrix units.
//
//   gate/up: G = acc_g * scale[row] * channel scale, U likewise, H = silu(G) * U (bf16)
//   down:    Y = acc * scale[row] * channel scale (bf16)
//
// |q| <= 127, so a sum over K <= 65536 stays below 2^30.1 and never wraps.
//
// Design (gfx950), after the bf16 kernel of grouped_gemm_lds.hip: 256 threads (four
// waves, one workgroup per CU), tiles of up to 256 rows x 256 weight channels (SwiGLU:
// 128 gate channels and the matching 128 up channels), four LDS stages of K = 64 filled
// by buffer_load ... lds three stages ahead, v_mfma_i32_32x32x32_i8 with every LDS read
// and DMA load issued in the shadow of an MFMA. What differs: both operands are stored
// K-contiguous in blocks of 64 (one stage = 64 bytes of a row), so both are read by
// ds_read_b128 with no transpose, and a stage of a tile is one contiguous run of HBM.
// The order of K inside a fragment is free as long as A and B agree; both take the
// bytes 16 * (lane / 32) .. + 15 of a 32-byte slice.
#include <type_traits>

#include "lds_pipe.h"

namespace moe {
namespace {

using namespace gemm;

typedef int i32x16_t __attribute__((ext_vector_type(16)));

constexpr int kBK = 64;       // K per stage, in elements and bytes
constexpr int kStages = 4;
constexpr uint32_t kAStageBytes = 256 * kBK;
constexpr uint32_t kBStageBytes = 256 * kBK;

struct Frags {
  i32x4_t a[4], b[4];  // 32-row (32-channel) blocks, 16 K bytes per lane
};

template <int IMM>
__device__ __forceinline__ i32x4_t ds_read_frag(uint32_t addr) {
  i32x4_t v;
  asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(IMM));
  return v;
}

// H rows of the tile (32, 64, 128 or 256), 256 weight channels.
template <int H>
struct Layout {
  static constexpr int WM = H >= 64 ? 2 : 1;  // waves along M
  static constexpr int WN = 4 / WM;
  static constexpr int MI = H / WM / 32;      // 32-row blocks per wave
  static constexpr int NI = 256 / WN / 32;    // 32-channel blocks per wave
  static constexpr int A_INSTR = H / 16;      // 1 KB loads per activation stage
  static constexpr int A_PER_WAVE = (A_INSTR + 3) / 4;
  static constexpr int B_PER_WAVE = 4;
  static constexpr int PER = A_PER_WAVE + B_PER_WAVE;
  static constexpr int READS = MI + NI;
  static constexpr int NMFMA = MI * NI;
};

// One tile: rows [row0, row0 + rows_valid) of A (K-blocks of n_rows rows), channels
// from n0 of the expert's weights.
template <bool SWIGLU, int H>
__device__ __forceinline__ void gemm_tile(char* smem, const uint8_t* __restrict__ A, const float* __restrict__ a_scale,
                                          const uint8_t* __restrict__ Bexp, const float* __restrict__ b_scale,
                                          uint16_t* __restrict__ C, int row0, int rows_valid, int n0, int ksteps, int N,
                                          int64_t n_rows) {
  using L = Layout<H>;
  constexpr int MI = L::MI, NI = L::NI, WN = L::WN, PER = L::PER, NS = kStages;
  const int tid = threadIdx.x;
  const int lane = lane_id();
  const int wave = uniform(tid / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int l31 = lane & 31;
  const int64_t channels = SWIGLU ? 2 * static_cast<int64_t>(N) : N;

  const uint32_t sA = uniform(static_cast<int>(lds_addr(smem)));
  const uint32_t sB = sA + NS * kAStageBytes;

  // Load j of a stage covers rows 16 j .. 16 j + 15: lane L brings row 16 j + L / 4, chunk
  // (L & 3) ^ ((row >> 2) & 3) into LDS slot L, so that 16 consecutive rows of a fragment
  // read fall into 16 distinct bank groups. Rows past the end read zeros.
  const uint32_t chunk = static_cast<uint32_t>((lane & 3) ^ ((lane >> 4) & 3)) * 16u;
  uint32_t a_voff[L::A_PER_WAVE], b_voff[L::B_PER_WAVE];
  int a_slot[L::A_PER_WAVE];
#pragma unroll
  for (int jj = 0; jj < L::A_PER_WAVE; ++jj) {
    const int j = (wave * L::A_PER_WAVE + jj) % L::A_INSTR;
    a_slot[jj] = j;
    a_voff[jj] = static_cast<uint32_t>(16 * j + (lane >> 2)) * 64u + chunk;
  }
#pragma unroll
  for (int jj = 0; jj < L::B_PER_WAVE; ++jj) {
    const int r = 16 * (wave * L::B_PER_WAVE + jj) + (lane >> 2);  // row of the weight stage
    const int c = SWIGLU ? n0 + (r & 127) : n0 + r;
    // channels past N point past the buffer: zeros, without a fetch
    b_voff[jj] = c < N ? static_cast<uint32_t>(c + (SWIGLU && r >= 128 ? N : 0)) * 64u + chunk : 0x80000000u;
  }
  const uint8_t* a_tile = A + static_cast<int64_t>(row0) * 64;

  uint32_t a_rd[2], b_rd[2];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    const uint32_t c = static_cast<uint32_t>((2 * kk + (lane >> 5)) ^ ((l31 >> 2) & 3)) * 16u;
    a_rd[kk] = static_cast<uint32_t>(wm * (MI * 32) + l31) * 64u + c;
    // gate blocks first, the up half 128 rows further on
    b_rd[kk] = static_cast<uint32_t>(wn * (SWIGLU ? 128 / WN : 256 / WN) + l31) * 64u + c;
  }
  constexpr int R = L::READS, NM = L::NMFMA;
  auto read_one = [&](Frags& f, int buf, auto kk_c, auto r_c) {
    constexpr int kk = decltype(kk_c)::value, r = decltype(r_c)::value;
    if constexpr (r < MI) {
      f.a[r] = ds_read_frag<r * 2048>(sA + buf * kAStageBytes + a_rd[kk]);
    } else {
      constexpr int ni = r - MI;
      constexpr int off = SWIGLU ? (ni < NI / 2 ? ni * 2048 : 128 * 64 + (ni - NI / 2) * 2048) : ni * 2048;
      f.b[ni] = ds_read_frag<off>(sB + buf * kBStageBytes + b_rd[kk]);
    }
  };
  auto tie_frags = [&](Frags& f) {
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) tie(f.a[mi]);
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) tie(f.b[ni]);
  };

  i32x16_t acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[mi][ni][r] = 0;

  auto mfma_one = [&](const Frags& f, auto q_c) {
    constexpr int q = decltype(q_c)::value, mi = q / NI, ni = q % NI;
    acc[mi][ni] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.a[mi], f.b[ni], acc[mi][ni], 0, 0, 0);
  };

  struct StageLoads {
    __amdgpu_buffer_rsrc_t ra, rb;
    uint32_t la, lb;
  };
  auto stage_loads = [&](int s) {
    const int buf = s % NS;
    return StageLoads{make_rsrc(a_tile + static_cast<int64_t>(s) * n_rows * 64, static_cast<uint32_t>(rows_valid) * 64u),
                      make_rsrc(Bexp + static_cast<int64_t>(s) * channels * 64, static_cast<uint32_t>(channels) * 64u),
                      sA + buf * kAStageBytes, sB + buf * kBStageBytes};
  };
  auto dma_one = [&](const StageLoads& st, auto j_c) {
    constexpr int j = decltype(j_c)::value;
    if constexpr (j < L::A_PER_WAVE) dma16(st.ra, a_voff[j], st.la + a_slot[j] * 1024);
    else dma16(st.rb, b_voff[j - L::A_PER_WAVE], st.lb + (wave * L::B_PER_WAVE + (j - L::A_PER_WAVE)) * 1024);
  };

  // Stage s lands in buffer s % NS, issued NS - 1 stages ahead; when a wave waits for
  // stage s, min(NS - 2, ksteps - 1 - s) later stages of its own loads may be in flight.
  auto wait_stage = [&](int s) {
    const int after = min(NS - 2, ksteps - 1 - s);
    if (after >= 2) wait_vmcnt<2 * PER>();
    else if (after == 1) wait_vmcnt<PER>();
    else wait_vmcnt<0>();
  };
  using K0 = std::integral_constant<int, 0>;
  using K1 = std::integral_constant<int, 1>;

  // One stage: slice 0 (fragments f0) carries slice 1's reads, then the stage barrier;
  // slice 1 carries the next stage's slice-0 reads and the loads of stage ks + NS.
  Frags f0, f1;
  auto stage = [&](int ks, auto dma_c, auto more_c) {
    constexpr bool DMA = decltype(dma_c)::value, MORE = decltype(more_c)::value;
    const int buf = ks % NS;
    wait_lgkmcnt<0>();
    tie_frags(f0);
    __builtin_amdgcn_sched_barrier(0);
    static_for<0, NM>([&](auto q) {
      mfma_one(f0, q);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (decltype(q)::value < R) read_one(f1, buf, K1{}, q);
      __builtin_amdgcn_sched_barrier(0);
    });
    static_for<(NM < R ? NM : R), R>([&](auto r) { read_one(f1, buf, K1{}, r); });
    wait_lgkmcnt<0>();  // this wave's reads of stage ks are complete
    tie_frags(f1);
    if constexpr (MORE) {
      wait_stage(ks + 1);
      __builtin_amdgcn_s_barrier();  // stage ks + 1 landed for every wave; nobody reads stage ks any more
    }
    __builtin_amdgcn_sched_barrier(0);
    StageLoads st;
    if constexpr (DMA) st = stage_loads(ks + NS);
    const int nbuf = (ks + 1) % NS;
    static_for<0, NM>([&](auto q_c) {
      constexpr int q = decltype(q_c)::value;
      mfma_one(f1, q_c);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (MORE && q < R) read_one(f0, nbuf, K0{}, q_c);
      if constexpr (DMA && q % 2 == 0 && q / 2 < PER) dma_one(st, std::integral_constant<int, q / 2>{});
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (MORE) static_for<(NM < R ? NM : R), R>([&](auto r) { read_one(f0, nbuf, K0{}, r); });
    if constexpr (DMA) static_for<((NM + 1) / 2 < PER ? (NM + 1) / 2 : PER), PER>([&](auto j) { dma_one(st, j); });
    __builtin_amdgcn_sched_barrier(0);
  };

  for (int s = 0; s < NS - 1 && s < ksteps; ++s) {
    const StageLoads st = stage_loads(s);
    static_for<0, PER>([&](auto j) { dma_one(st, j); });
  }
  wait_stage(0);
  __builtin_amdgcn_s_barrier();
  if (NS - 1 < ksteps) {
    const StageLoads st = stage_loads(NS - 1);
    static_for<0, PER>([&](auto j) { dma_one(st, j); });
  }
  static_for<0, R>([&](auto r) { read_one(f0, 0, K0{}, r); });
  int ks = 0;
  for (; ks + NS < ksteps; ++ks) stage(ks, std::true_type{}, std::true_type{});
  for (; ks + 1 < ksteps; ++ks) stage(ks, std::false_type{}, std::true_type{});
  stage(ks, std::false_type{}, std::false_type{});

  // ---- epilogue: scales in fp32, one rounding to bf16, stores bounded by the valid rows ----
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(a_scale + row0, static_cast<uint32_t>(rows_valid) * 4u);
  const __amdgpu_buffer_rsrc_t rc =
      make_rsrc(C + static_cast<int64_t>(row0) * N, static_cast<uint32_t>(rows_valid) * static_cast<uint32_t>(N) * 2u);
  constexpr int NO = SWIGLU ? NI / 2 : NI;  // output blocks per wave
  uint32_t coff[NO];
  float sb[NI];
#pragma unroll
  for (int ni = 0; ni < NO; ++ni) {
    const int col = n0 + wn * (SWIGLU ? 128 / WN : 256 / WN) + ni * 32 + l31;
    coff[ni] = col < N ? static_cast<uint32_t>(col) * 2u : 0x80000000u;
    sb[ni] = col < N ? b_scale[col] : 0.f;
    if (SWIGLU) sb[ni + NO] = col < N ? b_scale[N + col] : 0.f;
  }
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = wm * (MI * 32) + mi * 32 + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3);
      const float sa = __uint_as_float(
          static_cast<uint32_t>(__builtin_amdgcn_raw_buffer_load_b32(rs, row * 4, 0, 0)));
#pragma unroll
      for (int ni = 0; ni < NO; ++ni) {
        float v;
        if constexpr (SWIGLU) {
          const float g = static_cast<float>(acc[mi][ni][r]) * sb[ni] * sa;
          const float u = static_cast<float>(acc[mi][ni + NO][r]) * sb[ni + NO] * sa;
          v = silu_fast(g) * u;
        } else {
          v = static_cast<float>(acc[mi][ni][r]) * sb[ni] * sa;
        }
        const __bf16 o = static_cast<__bf16>(v);
        __builtin_amdgcn_raw_buffer_store_b16(
            __builtin_bit_cast(unsigned short, o), rc,
            static_cast<int>(static_cast<uint32_t>(row) * static_cast<uint32_t>(N) * 2u + coff[ni]), 0, 0);
      }
    }
}

template <bool SWIGLU>
__global__ __launch_bounds__(kThreads, 1) void grouped_gemm_int8_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ a_scale, const uint8_t* __restrict__ B,
    const float* __restrict__ b_scale, uint16_t* __restrict__ C, const int32_t* __restrict__ offsets, int e_begin,
    int e_loc, int kblocks, int N, int n_max) {
  __shared__ __attribute__((aligned(1024))) char smem[kStages * (kAStageBytes + kBStageBytes)];
  __shared__ SortedTileMap tm;
  build_sorted_tile_map<256, 0>(tm, offsets, e_begin, e_loc, n_max);
  constexpr int kOutCols = SWIGLU ? 128 : 256;
  const int n_tiles = (N + kOutCols - 1) / kOutCols;
  const int total = uniform(tm.mstart[e_loc]) * n_tiles;
  const int64_t channels = SWIGLU ? 2 * static_cast<int64_t>(N) : N;
  const int G = gridDim.x, r = xcd_remap(blockIdx.x, G);
  for (int i = 0;; ++i) {
    const int tile = snake_tile(i, r, G);
    if (tile >= total) break;
    const SortedTile tc = find_sorted_tile(tm, tile, n_tiles, e_loc);
    const int row0 = uniform(tm.rstart[tc.e]) + tc.mt * 256;
    const int row_end = uniform(tm.rstart[tc.e + 1]);
    const int rows = min(row_end - row0, 256);
    const int n0 = tc.nt * kOutCols;
    const uint8_t* Be = B + tc.e * channels * kblocks * 64;
    const float* be = b_scale + tc.e * channels;
    if (rows > 128) gemm_tile<SWIGLU, 256>(smem, A, a_scale, Be, be, C, row0, rows, n0, kblocks, N, n_max);
    else if (rows > 64) gemm_tile<SWIGLU, 128>(smem, A, a_scale, Be, be, C, row0, rows, n0, kblocks, N, n_max);
    else if (rows > 32) gemm_tile<SWIGLU, 64>(smem, A, a_scale, Be, be, C, row0, rows, n0, kblocks, N, n_max);
    else gemm_tile<SWIGLU, 32>(smem, A, a_scale, Be, be, C, row0, rows, n0, kblocks, N, n_max);
    // every wave has waited for its last LDS reads; the next tile's loads may land
    __builtin_amdgcn_s_barrier();
  }
}

}  // namespace

hipError_t launch_grouped_gemm_int8(const void* a, const float* a_scale, const void* w, const float* w_scale, void* c,
                                    const int32_t* offsets, int e_begin, int e_loc, int K, int N, int64_t n_max,
                                    bool swiglu, hipStream_t stream) {
  const int cols = swiglu ? 128 : 256;
  const int grid = grouped_gemm_grid(n_max, e_loc, (N + cols - 1) / cols);
  const int kblocks = int8_kblocks(K);
  if (swiglu)
    hipLaunchKernelGGL(grouped_gemm_int8_kernel<true>, dim3(grid), dim3(kThreads), 0, stream,
                       static_cast<const uint8_t*>(a), a_scale, static_cast<const uint8_t*>(w), w_scale,
                       static_cast<uint16_t*>(c), offsets, e_begin, e_loc, kblocks, N, static_cast<int>(n_max));
  else
    hipLaunchKernelGGL(grouped_gemm_int8_kernel<false>, dim3(grid), dim3(kThreads), 0, stream,
                       static_cast<const uint8_t*>(a), a_scale, static_cast<const uint8_t*>(w), w_scale,
                       static_cast<uint16_t*>(c), offsets, e_begin, e_loc, kblocks, N, static_cast<int>(n_max));
  return hipGetLastError();
}

}  // namespace moe
