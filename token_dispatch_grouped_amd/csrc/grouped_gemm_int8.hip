// Grouped expert GEMM in 8-bit integers: the experts' SwiGLU FFN on quantised rows
// and weights (int8_rows.hip), with exact int32 sums on the matrix units.
//
//   gate/up: G = acc_g * scale[row] * channel scale, U likewise, H = silu(G) * U (bf16)
//   down:    Y = acc * scale[row] * channel scale (bf16)
//
// |q| <= 127, so a sum over K <= 65536 stays below 2^30.1 and never wraps.
//
// Design (gfx950): 256 threads (four waves), tiles of BM rows x 256 weight channels
// (SwiGLU: 128 gate channels and the matching 128 up channels), LDS stages of K = 64
// filled by buffer_load ... lds ahead of their use, v_mfma_i32_32x32x32_i8 with every
// LDS read and DMA load issued in the shadow of an MFMA. Both operands are stored
// K-contiguous in blocks of 64 (one stage = 64 bytes of a row), so both are read by
// ds_read_b128 with no transpose, and a stage of a tile is one contiguous run of HBM.
// The order of K inside a fragment is free as long as A and B agree; both take the
// bytes 16 * (lane / 32) .. + 15 of a 32-byte slice.
//
// Two shapes of workgroup (int8_tile_rows says when; two more, for few rows, are in int8_few.hip):
//   tall   BM = 256 (288 where a remainder of up to 32 rows rides along), one workgroup
//          per CU with all of its LDS: five stages (four with 288 rows). For experts with
//          many rows: each byte brought to a CU is used by the most products.
//   short  BM = 128, two workgroups per CU: one computes or waits while the other's
//          loads are in flight. For few rows per expert, where the weight stream bounds.
// Tiles are listed once per call by plan_tiles (int8_rows.hip's first launch).
#include <type_traits>

#include "int8_plan.h"
#include "lds_pipe.h"

namespace moe {
namespace {

using namespace gemm;
using int8::RowGroup;

typedef int i32x16_t __attribute__((ext_vector_type(16)));

constexpr int kBK = 64;  // K per stage, in elements and bytes
constexpr int kTallLds = 160 * 1024;
constexpr int kShortLds = 72 * 1024;

struct Frags {
  i32x4_t a[5], b[4];  // 32-row (32-channel) blocks, 16 K bytes per lane; a[MI]: the extra block of 288 rows
};

template <int IMM>
__device__ __forceinline__ i32x4_t ds_read_frag(uint32_t addr) {
  i32x4_t v;
  asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(IMM));
  return v;
}

// c += a * b with c held in VGPRs (the accumulator file is full)
__device__ __forceinline__ void mfma_i8_in_vgprs(i32x16_t& c, const i32x4_t& a, const i32x4_t& b) {
  asm volatile("v_mfma_i32_32x32x32_i8 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
}

// H rows of the tile: 32, 64, 128, 256 or 288; BN weight channels: 256, or 128 for half of a
// tall tile. A 288-row tile is a 256-row tile plus one 32-row block that every wave shares,
// each computing it against half of its own channel blocks (all of its two at BN = 128,
// where the second wave row's results are the first's and are not stored).
template <int H, int BN, int LDS>
struct Layout {
  static constexpr int WM = H >= 64 ? 2 : 1;  // waves along M
  static constexpr int WN = 4 / WM;
  static constexpr int MI = H / WM / 32;      // 32-row blocks per wave (regular part)
  static constexpr int NI = BN / WN / 32;     // 32-channel blocks per wave
  static constexpr int XR = H == 288 ? 1 : 0;
  static constexpr int MX = 2 * XR;           // extra MFMAs per wave and slice
  static constexpr int A_INSTR = H / 16;      // 1 KB loads per activation stage
  static constexpr int A_PER_WAVE = (A_INSTR + 3) / 4;
  static constexpr int B_PER_WAVE = BN / 64;
  static constexpr int PER = A_PER_WAVE + B_PER_WAVE;
  static constexpr int READS = MI + XR + NI;
  static constexpr int NMFMA = MX + MI * NI;
  static constexpr uint32_t A_BYTES = H * kBK, B_BYTES = BN * kBK;
  // stages that fit, at most six (vmcnt counts 63 loads, a wave has PER per stage)
  static constexpr int FIT = LDS / static_cast<int>(A_BYTES + B_BYTES);
  static constexpr int NS = FIT < 6 ? FIT : 6;
  static_assert((NS - 2) * PER < 64, "loads in flight are counted in six bits");
  static_assert(BN == 256 || (BN == 128 && WN == 2), "half-width tiles have two waves along N");
};

// One tile: rows [row0, row0 + rows_valid) of A (K-blocks of n_rows rows), channels
// from n0 of the expert's weights. STREAM: no other row tile reads this weight panel.
template <bool SWIGLU, int H, int BN, int LDS, bool STREAM>
__device__ __forceinline__ void gemm_tile(char* smem, const uint8_t* __restrict__ A, const float* __restrict__ a_scale,
                                          const uint8_t* __restrict__ Bexp, const float* __restrict__ b_scale,
                                          uint16_t* __restrict__ C, int row0, int rows_valid, int n0, int ksteps, int N,
                                          int64_t n_rows) {
  using L = Layout<H, BN, LDS>;
  constexpr int HB = BN / 2;
  constexpr int MI = L::MI, NI = L::NI, WM = L::WM, WN = L::WN, PER = L::PER, NS = L::NS;
  // opaque: the lane's offsets are recomputed for each tile instead of living through the kernel for every height
  const int tid = opaque(static_cast<int>(threadIdx.x));
  const int lane = tid & (kWave - 1);
  const int wave = uniform(tid / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int l31 = lane & 31;
  const int64_t channels = SWIGLU ? 2 * static_cast<int64_t>(N) : N;

  const uint32_t sA = uniform(static_cast<int>(lds_addr(smem)));
  const uint32_t sB = sA + NS * L::A_BYTES;

  // Load j of a stage covers rows 16 j .. 16 j + 15: lane L brings row 16 j + L / 4, chunk
  // (L & 3) ^ ((row >> 2) & 3) into LDS slot L, so that 16 consecutive rows of a fragment
  // read fall into 16 distinct bank groups. Rows past the end read zeros.
  const uint32_t chunk = static_cast<uint32_t>((lane & 3) ^ ((lane >> 4) & 3)) * 16u;
  uint32_t a_voff[L::A_PER_WAVE], b_voff[L::B_PER_WAVE];
  int a_slot[L::A_PER_WAVE];
#pragma unroll
  for (int jj = 0; jj < L::A_PER_WAVE; ++jj) {
    // slots beyond A_INSTR repeat an earlier one (identical bytes to the same place)
    const int j = (wave * L::A_PER_WAVE + jj) % L::A_INSTR;
    a_slot[jj] = j;
    a_voff[jj] = static_cast<uint32_t>(16 * j + (lane >> 2)) * 64u + chunk;
  }
#pragma unroll
  for (int jj = 0; jj < L::B_PER_WAVE; ++jj) {
    const int r = 16 * (wave * L::B_PER_WAVE + jj) + (lane >> 2);  // row of the weight stage
    const int c = SWIGLU ? n0 + (r & (HB - 1)) : n0 + r;
    // channels past N point past the buffer: zeros, without a fetch
    b_voff[jj] = c < N ? static_cast<uint32_t>(c + (SWIGLU && r >= HB ? N : 0)) * 64u + chunk : 0x80000000u;
  }
  const uint8_t* a_tile = A + static_cast<int64_t>(row0) * 64;
  // these threads' row scales, for the epilogue (asked for before the pipeline's loads, so no wait counts them)
  const float my_scale = tid < rows_valid ? a_scale[row0 + tid] : 0.f;
  const float my_scale_x = L::XR && tid < 32 && 256 + tid < rows_valid ? a_scale[row0 + 256 + tid] : 0.f;

  // Channel block of register slot ni, in rows of the weight stage (SwiGLU: slots [0, NI/2)
  // gate, the rest the matching up blocks). In a 288-row tile the second wave row holds its
  // blocks in swapped slots, so that every wave's share of the extra row block is slot 0 (with
  // SwiGLU and its up pair, else and slot 1), the blocks that the other wave row does not take.
  constexpr int X1 = SWIGLU ? NI / 2 : 1;
  auto bcol = [&](int ni) {
    if (L::XR && wm && BN == 256) ni = SWIGLU ? ni ^ 1 : ni ^ 2;
    if (SWIGLU) return ni < NI / 2 ? wn * (HB / WN) + ni * 32 : HB + wn * (HB / WN) + (ni - NI / 2) * 32;
    return wn * (BN / WN) + ni * 32;
  };
  uint32_t a_rd[2], b_rd[2], b_slot[NI];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    const uint32_t c = static_cast<uint32_t>((2 * kk + (lane >> 5)) ^ ((l31 >> 2) & 3)) * 16u;
    a_rd[kk] = static_cast<uint32_t>(wm * (MI * 32) + l31) * 64u + c;
    b_rd[kk] = static_cast<uint32_t>(l31) * 64u + c;
  }
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) b_slot[ni] = static_cast<uint32_t>(bcol(ni)) * 64u;
  constexpr int R = L::READS, NM = L::NMFMA;
  auto read_one = [&](Frags& f, int buf, auto kk_c, auto r_c) {
    constexpr int kk = decltype(kk_c)::value, r = decltype(r_c)::value;
    if constexpr (r < MI) {
      f.a[r] = ds_read_frag<r * 2048>(sA + buf * L::A_BYTES + a_rd[kk]);
    } else if constexpr (r < MI + L::XR) {
      f.a[MI] = ds_read_frag<0>(sA + buf * L::A_BYTES + a_rd[kk] - wm * (MI * 2048u) + WM * MI * 2048u);
    } else {
      constexpr int ni = r - MI - L::XR;
      f.b[ni] = ds_read_frag<0>(sB + buf * L::B_BYTES + b_slot[ni] + b_rd[kk]);
    }
  };
  auto tie_frags = [&](Frags& f) {
#pragma unroll
    for (int mi = 0; mi < MI + L::XR; ++mi) tie(f.a[mi]);
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) tie(f.b[ni]);
  };

  i32x16_t acc[MI][NI], acc_x[L::MX > 0 ? L::MX : 1];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[mi][ni][r] = 0;
#pragma unroll
  for (int x = 0; x < L::MX; ++x)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc_x[x][r] = 0;

  // MFMA number q of a slice: first this wave's share of the extra row block (its results,
  // written outside the compiler's view, are next read at least NMFMA - MX MFMAs later)
  auto mfma_one = [&](const Frags& f, auto q_c) {
    constexpr int q = decltype(q_c)::value;
    if constexpr (q < L::MX) {
      mfma_i8_in_vgprs(acc_x[q], f.a[MI], f.b[q == 0 ? 0 : X1]);
    } else {
      constexpr int mi = (q - L::MX) / NI, ni = (q - L::MX) % NI;
      acc[mi][ni] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.a[mi], f.b[ni], acc[mi][ni], 0, 0, 0);
    }
  };

  struct StageLoads {
    __amdgpu_buffer_rsrc_t ra, rb;
    uint32_t la, lb;
  };
  auto stage_loads = [&](int s) {
    const int buf = s % NS;
    return StageLoads{make_rsrc(a_tile + static_cast<int64_t>(s) * n_rows * 64, static_cast<uint32_t>(rows_valid) * 64u),
                      make_rsrc(Bexp + static_cast<int64_t>(s) * channels * 64, static_cast<uint32_t>(channels) * 64u),
                      sA + buf * L::A_BYTES, sB + buf * L::B_BYTES};
  };
  auto dma_one = [&](const StageLoads& st, auto j_c) {
    constexpr int j = decltype(j_c)::value;
    if constexpr (j < L::A_PER_WAVE) dma16(st.ra, a_voff[j], st.la + a_slot[j] * 1024);
    else
      dma16<STREAM ? kCpolNT : 0>(st.rb, b_voff[j - L::A_PER_WAVE],
                                  st.lb + (wave * L::B_PER_WAVE + (j - L::A_PER_WAVE)) * 1024);
  };

  // Stage s lands in buffer s % NS, issued NS - 1 stages ahead; when a wave waits for
  // stage s, min(NS - 2, ksteps - 1 - s) later stages of its own loads may be in flight.
  auto wait_stage = [&](int s) {
    const int after = min(NS - 2, ksteps - 1 - s);
    bool done = false;
    static_for<0, NS - 2>([&](auto i) {
      constexpr int n = NS - 2 - decltype(i)::value;  // NS - 2 .. 1
      if (!done && after >= n) {
        wait_vmcnt<n * PER>();
        done = true;
      }
    });
    if (!done) wait_vmcnt<0>();
  };
  using K0 = std::integral_constant<int, 0>;
  using K1 = std::integral_constant<int, 1>;

  // One stage: slice 0 (fragments f0) carries slice 1's reads, then the stage barrier;
  // slice 1 carries the next stage's slice-0 reads and the loads of stage ks + NS.
  Frags f0, f1;
  int buf = 0;  // ks % NS
  auto stage = [&](int ks, auto dma_c, auto more_c) {
    constexpr bool DMA = decltype(dma_c)::value, MORE = decltype(more_c)::value;
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
    const int nbuf = buf + 1 == NS ? 0 : buf + 1;
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
    buf = nbuf;
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
  // The row scales pass through LDS, in the activation buffer that the last stages left
  // untouched (stage ksteps - NS's, free since its barrier).
  float* row_scale = reinterpret_cast<float*>(smem + (ksteps % NS) * L::A_BYTES);
  if (tid < H) row_scale[tid] = my_scale;
  if (L::XR && tid < 32) row_scale[256 + tid] = my_scale_x;
  __syncthreads();
  const __amdgpu_buffer_rsrc_t rc =
      make_rsrc(C + static_cast<int64_t>(row0) * N, static_cast<uint32_t>(rows_valid) * static_cast<uint32_t>(N) * 2u);
  constexpr int NO = SWIGLU ? NI / 2 : NI;  // output blocks per wave
  uint32_t coff[NO];
  float sb[NI];
#pragma unroll
  for (int ni = 0; ni < NO; ++ni) {
    const int col = n0 + bcol(ni) + l31;
    coff[ni] = col < N ? static_cast<uint32_t>(col) * 2u : 0x80000000u;
    sb[ni] = col < N ? b_scale[col] : 0.f;
    if (SWIGLU) sb[ni + NO] = col < N ? b_scale[N + col] : 0.f;
  }
  auto emit = [&](int g, int u, float sg, float su, float sa, int row, uint32_t co) {
    float v;
    if constexpr (SWIGLU) {
      const float gate = static_cast<float>(g) * sg * sa;
      v = silu_fast(gate) * (static_cast<float>(u) * su * sa);
    } else {
      v = static_cast<float>(g) * sg * sa;
    }
    const __bf16 o = static_cast<__bf16>(v);
    __builtin_amdgcn_raw_buffer_store_b16(
        __builtin_bit_cast(unsigned short, o), rc,
        static_cast<int>(static_cast<uint32_t>(row) * static_cast<uint32_t>(N) * 2u + co), 0, 0);
  };
#pragma unroll
  for (int mi = 0; mi < MI + L::XR; ++mi)
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const bool x = mi == MI;  // the extra row block
      const int row4 = (x ? WM * MI * 32 : wm * (MI * 32) + mi * 32) + r4 * 8 + (lane >> 5) * 4;  // rows row4 .. + 3
      const float4 sa4 = *reinterpret_cast<const float4*>(row_scale + row4);
      const float sa[4] = {sa4.x, sa4.y, sa4.z, sa4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 4 * r4 + j;
        if (x) {
          if (BN == 128 && wm != 0) continue;  // the first wave row stores the shared block
          if constexpr (L::XR) {
            if constexpr (SWIGLU) {
              emit(acc_x[0][r], acc_x[1][r], sb[0], sb[NO], sa[j], row4 + j, coff[0]);
            } else {
              emit(acc_x[0][r], 0, sb[0], 0.f, sa[j], row4 + j, coff[0]);
              emit(acc_x[1][r], 0, sb[1], 0.f, sa[j], row4 + j, coff[1]);
            }
          }
        } else {
#pragma unroll
          for (int ni = 0; ni < NO; ++ni)
            emit(acc[mi < MI ? mi : 0][ni][r], SWIGLU ? acc[mi < MI ? mi : 0][SWIGLU ? ni + NO : 0][r] : 0, sb[ni],
                 SWIGLU ? sb[SWIGLU ? ni + NO : 0] : 0.f, sa[j], row4 + j, coff[ni]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // a few rows at a time: the accumulators leave no room for more
    }
}

template <bool SWIGLU, bool TALL>
__global__ __launch_bounds__(kThreads, TALL ? 1 : 2) void grouped_gemm_int8_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ a_scale, const uint8_t* __restrict__ B,
    const float* __restrict__ b_scale, uint16_t* __restrict__ C, const int* __restrict__ n_row_tiles,
    const RowGroup* __restrict__ groups, int kblocks, int N, int64_t n_max) {
  // n_row_tiles[0]: all entries, [1]: those of experts with tall tiles (they come first)
  constexpr int LDS = TALL ? kTallLds : kShortLds;
  constexpr int BM = TALL ? int8::kTallRows : int8::kShortRows;
  __shared__ __attribute__((aligned(1024))) char smem[LDS];
  constexpr int kOutCols = SWIGLU ? 128 : 256;
  const int n_tiles = (N + kOutCols - 1) / kOutCols;
  const int total = uniform(*n_row_tiles) * n_tiles;
  const int64_t channels = SWIGLU ? 2 * static_cast<int64_t>(N) : N;
  const int G = gridDim.x, per = G >> 3;
  const bool spread = (G & 7) == 0;
  const int r = xcd_remap(blockIdx.x, G);
  // The last, partial round: where its tall tiles can be halved and all of it still fits one
  // round, they are (16 experts of 256 rows, 2880 x 2880: gate/up is 368 tiles on 256 CUs).
  const int rounds = (total + G - 1) / G, last = total - (rounds - 1) * G;
  const int tall_last = min(max(uniform(n_row_tiles[1]) * n_tiles - (rounds - 1) * G, 0), last);
  const int n_split = TALL && last < G && last + tall_last <= G ? tall_last : 0;
  for (int i = 0;; ++i) {
    // Whole rounds give each XCD a contiguous run of tile ids, forward and backward in turn. The
    // last, partial one deals its tiles evenly over the XCDs: each has its own way to HBM, and
    // on 3.5 of the 8 a half-full round took as long as a full one (16 experts of 256 rows,
    // 2880 x 2880: gate/up 98 -> 90 us).
    int tile, half = 0;  // half: 0 the whole tile, 1 or 2 its first or second half
    const int rest = total - i * G;
    if (rest >= G) {
      tile = snake_tile(i, r, G);
    } else {
      const int items = rest + n_split;
      int lo = 0, j = r, hi = items;
      if (spread) {
        const int x = r / per;
        lo = items * x / 8;
        hi = items * (x + 1) / 8;
        j = r - x * per;
      }
      if (rest <= 0 || lo + j >= hi) break;
      const int item = lo + j;
      tile = i * G + (item < 2 * n_split ? item >> 1 : item - n_split);
      if (item < 2 * n_split) half = 1 + (item & 1);
    }
    // ids of a group of row tiles of one expert: row tile fastest, then the column block
    const int q = tile / n_tiles;
    const RowGroup g = groups[q];
    const int off = tile - (q - uniform(g.index)) * n_tiles;
    const int in_group = uniform(g.tiles);
    const int mt = off % in_group, n0 = off / in_group * kOutCols + (half == 2 ? kOutCols / 2 : 0);
    if (n0 >= N) break;  // the second half of a last column block that has only a first
    const int row0 = uniform(g.row0) + mt * BM;
    const int rows = uniform(g.last) && mt == in_group - 1 ? uniform(g.row_end) - row0 : BM;
    const int e = uniform(g.expert);
    const uint8_t* Be = B + e * channels * kblocks * 64;
    const float* be = b_scale + e * channels;
    // An expert with one row tile reads each weight panel once: streamed past the caches.
    // (128 experts of one row, 2880 x 2880: gate/up 400 -> 338 us; two row tiles of 128 that share
    // a panel took 530 MB instead of 265 from HBM with the same policy.)
    auto run = [&](auto stream) {
      constexpr bool S = decltype(stream)::value;
      if constexpr (TALL) {
        if (half) {
          if (rows > 256)
            return gemm_tile<SWIGLU, 288, 128, LDS, S>(smem, A, a_scale, Be, be, C, row0, rows, n0, kblocks, N, n_max);
          return gemm_tile<SWIGLU, 256, 128, LDS, S>(smem, A, a_scale, Be, be, C, row0, rows, n0, kblocks, N, n_max);
        }
        if (rows > 256)
          return gemm_tile<SWIGLU, 288, 256, LDS, S>(smem, A, a_scale, Be, be, C, row0, rows, n0, kblocks, N, n_max);
        if (rows > 128)
          return gemm_tile<SWIGLU, 256, 256, LDS, S>(smem, A, a_scale, Be, be, C, row0, rows, n0, kblocks, N, n_max);
      }
      if (rows > 64)
        return gemm_tile<SWIGLU, 128, 256, LDS, S>(smem, A, a_scale, Be, be, C, row0, rows, n0, kblocks, N, n_max);
      if (rows > 32)
        return gemm_tile<SWIGLU, 64, 256, LDS, S>(smem, A, a_scale, Be, be, C, row0, rows, n0, kblocks, N, n_max);
      return gemm_tile<SWIGLU, 32, 256, LDS, S>(smem, A, a_scale, Be, be, C, row0, rows, n0, kblocks, N, n_max);
    };
    if (uniform(g.alone)) run(std::true_type{});
    else run(std::false_type{});
    // every wave has waited for its last LDS reads; the next tile's loads may land
    __builtin_amdgcn_s_barrier();
  }
}

}  // namespace

hipError_t launch_grouped_gemm_int8(const void* a, const float* a_scale, const void* w, const float* w_scale, void* c,
                                    const void* plan, int tile_rows, int e_loc, int K, int N, int64_t n_max,
                                    bool swiglu, hipStream_t stream) {
  if (tile_rows == int8::kThinRows)
    return launch_int8_thin(a, a_scale, w, w_scale, c, plan, e_loc, K, N, n_max, swiglu, stream);
  const bool tall = tile_rows == int8::kTallRows;
  const int cols = swiglu ? 128 : 256;
  const int64_t tiles = int8::max_row_tiles(n_max, e_loc, tile_rows) * ((N + cols - 1) / cols);
  const int slots = device_cu_count() * (tall ? 1 : 2);
  const unsigned grid = static_cast<unsigned>(tiles < slots ? (tiles + 7) / 8 * 8 : slots);
  const int kblocks = int8_kblocks(K);
  const int* count = static_cast<const int*>(plan);
  const RowGroup* groups = reinterpret_cast<const RowGroup*>(static_cast<const char*>(plan) + int8::kPlanHeader);
#define MOE_INT8_GEMM(S, T)                                                                                          \
  hipLaunchKernelGGL((grouped_gemm_int8_kernel<S, T>), dim3(grid), dim3(kThreads), 0, stream,                        \
                     static_cast<const uint8_t*>(a), a_scale, static_cast<const uint8_t*>(w), w_scale,               \
                     static_cast<uint16_t*>(c), count, groups, kblocks, N, n_max)
  if (swiglu && tall) MOE_INT8_GEMM(true, true);
  else if (swiglu) MOE_INT8_GEMM(true, false);
  else if (tall) MOE_INT8_GEMM(false, true);
  else MOE_INT8_GEMM(false, false);
#undef MOE_INT8_GEMM
  return hipGetLastError();
}

}  // namespace moe
