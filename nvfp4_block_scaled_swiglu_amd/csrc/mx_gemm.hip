// mx_gemm.hip - MXFP4 product with FP32 accumulation and BF16 output (gfx950).
//
//   D[m, n] = RN_bf16(sum_k A[m, k] W[n, k]),  A, W = e2m1 * 2^(S - 127)
//
// The scaled matrix instructions take E2M1 codes and E8M0 scales as they are stored, so
// nothing is converted: 32x32x64 multiplies 32 rows by 32 columns over two blocks of 32,
// each lane giving the 16 code bytes and one scale byte of its (row, block). Every product
// is exact and the sums are fp32. The rate is four times that of fp16, so a K step has a
// quarter of the time to bring its operands that the fp16 form has per element.
#include <type_traits>

#include "mx.hpp"

namespace nvfp4 {

namespace {

typedef __attribute__((ext_vector_type(8))) int i32x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((address_space(3))) void lds_ptr_t;

struct MxGemmArgs {
  const uint8_t* aq;
  const uint8_t* as;
  const uint8_t* wq;
  const uint8_t* ws;
  uint16_t* d;
  int64_t ldd, m, n, k;
  int groups;            // scale columns / 4 = K steps of 128
  int tiles_m, tiles_n;
  int whole, parts;      // tiles [0, whole) are run whole, the rest in this many parts
  bool wide;             // D rows take 16-byte stores
};

__device__ __forceinline__ i32x8_t fp4_operand(const u32x4_t& c) {
  return i32x8_t{(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  bf16x2_t c;
  c[0] = (__bf16)lo;
  c[1] = (__bf16)hi;
  return as_u32(c);
}

// ---- tiles ---------------------------------------------------------------------------------
// A workgroup of 4 waves (2 x 2) computes (64 FM) x (64 FN), FM = FN = 4 for whole tiles; a
// wave owns FM x FN tiles of 32 x 32. A stage in LDS holds two K steps of 128: 128 code bytes
// a row, which a load instruction takes whole from 8 rows, and a KiB of scales per 128 rows.
// (64 bytes from 16 rows fetch every line twice: that took 37810 x 5376 x 14336 from 1,370 to
// 1,405 us, 1536 x 5376 x 14336 from 63.5 to 70.8.) Direct-to-LDS loads bring pair ps + kStages while pair
// ps is multiplied.
// A pair has four quarters of one MFMA per tile each: while the MFMAs of a quarter run, the
// fragments of the next are read from LDS, in a fixed order of fenced steps (left alone they
// gather in front of the MFMAs that use them, and one wave a SIMD waits for each). The
// barrier sits before the last quarter: every wave has then read all of the pair, whose
// stage takes the loads of pair ps + kStages, in this quarter and the first of the next pair;
// and each has seen its own loads of pair ps + 1 land.
constexpr int kWaves = 4;
constexpr int kBand = 8;  // M tiles per traversal band
constexpr int kCus = 256, kEdge = 256;

template <int FM, int FN>
struct Shape {
  static constexpr int kStages = FM * FN == 16 ? 2 : 3;  // a quarter with 2: 19.6 for 16.5 us, with 4 the same
  static constexpr int TM = 64 * FM, TN = 64 * FN;
  static constexpr int CodesA = TM * 128, CodesW = TN * 128;
  static constexpr int TilesA = TM / 128, Tiles = TilesA + TN / 128;   // of 128 rows of scales, 1 KiB each
  static constexpr int Stage = CodesA + CodesW + Tiles * 1024;
  static constexpr int LoadsA = CodesA / 1024 / kWaves, LoadsW = CodesW / 1024 / kWaves;
  static constexpr int Loads = LoadsA + LoadsW + 1;                 // the waves share the scale tiles
  static constexpr int RowBytes = 32 * FN * 2 + 16;                 // epilogue staging, padded
  static constexpr int Staging = kWaves * 32 * RowBytes;
  static constexpr int Lds = kStages * Stage > Staging ? kStages * Stage : Staging;
  static_assert(CodesA % (1024 * kWaves) == 0 && CodesW % (1024 * kWaves) == 0, "even code loads");
  static_assert((kStages - 1) * Loads < 64, "vmcnt immediate");
  static_assert(Tiles <= kWaves, "scale loads");
  static_assert((FM == 4 || FM == 2) && (FN == 4 || FN == 2), "scale reads");
};

// where 16-byte chunk c of row r lies in the row's 128 LDS bytes: the 16 rows that a phase of
// a fragment read meets (one chunk) then lie in different banks
__device__ __forceinline__ int chunk_at(int r, int c) { return c ^ ((r >> 1) & 7); }

__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// s_waitcnt vmcnt(n) lgkmcnt(15) expcnt(7)
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// the tile at rows m0, columns n0
template <int FM, int FN>
__device__ __forceinline__ void run_tile(const MxGemmArgs& a, int64_t m0, int64_t n0, uint8_t* smem) {
  using T = Shape<FM, FN>;
  constexpr int kStages = T::kStages;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int lr = lane & 31, h = lane >> 5;

  // Buffers of the tile's own rows: reads past them return zero.
  const int krow = (int)(a.k >> 1);
  const int rows_a = (int)(a.m - m0 < T::TM ? a.m - m0 : T::TM), rows_w = (int)(a.n - n0 < T::TN ? a.n - n0 : T::TN);
  const int srow = a.groups * 512;
  __amdgpu_buffer_rsrc_t rA =
      __builtin_amdgcn_make_buffer_rsrc((void*)(a.aq + m0 * krow), 0, rows_a * krow, 0x00020000);
  __amdgpu_buffer_rsrc_t rW =
      __builtin_amdgcn_make_buffer_rsrc((void*)(a.wq + n0 * krow), 0, rows_w * krow, 0x00020000);
  __amdgpu_buffer_rsrc_t rSA = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(a.as + (m0 >> 7) * srow), 0, ((rows_a + 127) >> 7) * srow, 0x00020000);
  __amdgpu_buffer_rsrc_t rSW = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(a.ws + (n0 >> 7) * srow), 0, ((rows_w + 127) >> 7) * srow, 0x00020000);

  // Load idx of this wave's share of pair ps. Code load j covers rows 8 j .. 8 j + 7; lane L
  // writes LDS bytes 16 L .. of that KiB, which hold chunk chunk_at(row, L & 7) (an
  // involution) of row 8 j + L / 8, or of the tile's last row behind it (results that are not
  // stored; cheaper than zeros). Chunks past K (and whole pairs past the last) read past the
  // buffer, where there is nothing but zeros.
  auto issue = [&](int ps, int stage, int idx) __attribute__((always_inline)) {
    uint8_t* st = smem + stage * T::Stage;
    if (idx < T::LoadsA + T::LoadsW) {
      const bool is_a = idx < T::LoadsA;
      const int j = wave + (is_a ? idx : idx - T::LoadsA) * kWaves;
      const int row = j * 8 + (lane >> 3);
      const int kb = ps * 128 + chunk_at(row, lane & 7) * 16, have = is_a ? rows_a : rows_w;
      const int off = kb < krow ? (row < have ? row : have - 1) * krow + kb : 0x7FFFFFF0;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? rA : rW, (lds_ptr_t*)(st + (is_a ? 0 : T::CodesA) + j * 1024), 16,
                                               off, 0, 0, 0);
    } else {
      const int q = wave % T::Tiles;  // some twice if there are fewer
      const bool is_a = q < T::TilesA;
      const int off = 2 * ps + (lane >> 5) < a.groups ? (is_a ? q : q - T::TilesA) * srow + ps * 1024 + lane * 16 : 0x7FFFFFF0;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? rSA : rSW, (lds_ptr_t*)(st + T::CodesA + T::CodesW + q * 1024), 16,
                                               off, 0, 0, 0);
    }
  };
  // quarter kk: lane half h takes block (chunk) 2 kk + h of the pair; fragment f of A, then W
  auto read_code = [&](int stage, int kk, int f, u32x4_t (&ca)[FM], u32x4_t (&cw)[FN]) __attribute__((always_inline)) {
    const uint8_t* st = smem + stage * T::Stage;
    const int c = 2 * kk + h;
    if (f < FM) {
      const int r = (wm * FM + f) * 32 + lr;
      ca[f] = *(const u32x4_t*)(st + r * 128 + chunk_at(r, c) * 16);
    } else {
      const int r = (wn * FN + f - FM) * 32 + lr;
      cw[f - FM] = *(const u32x4_t*)(st + T::CodesA + r * 128 + chunk_at(r, c) * 16);
    }
  };
  // the four scale bytes, of one step, of the rows of a side's fragments: 32-row groups lie
  // next to each other, so a lane's are one run
  auto read_scales = [&](int stage, int step, bool is_a, uint32_t (&sc)[FM + FN]) __attribute__((always_inline)) {
    const int g = is_a ? wm * FM : wn * FN, n = is_a ? FM : FN, at = is_a ? 0 : FM;
    const uint8_t* p = smem + stage * T::Stage + T::CodesA + T::CodesW + ((is_a ? 0 : T::TilesA) + (g >> 2)) * 1024 +
                       step * 512 + lr * 16 + (g & 3) * 4;
    if (n == 4) {
      const u32x4_t v = *(const u32x4_t*)p;
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[(at + i) % (FM + FN)] = v[i];
    } else {
      const u32x2_t v = *(const u32x2_t*)p;
      sc[at] = v[0];
      sc[at + 1] = v[1];
    }
  };

  constexpr int kEarly = T::Loads / 2;  // loads of a pair in the last quarter before it
  f32x16_t acc[FN][FM];
#pragma unroll
  for (int j = 0; j < FN; ++j)
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;

#pragma unroll
  for (int s = 0; s < kStages; ++s)
#pragma unroll
    for (int idx = 0; idx < (s + 1 < kStages ? T::Loads : kEarly); ++idx) issue(s, s, idx);
  wait_loads<(kStages - 2) * T::Loads + kEarly>();
  barrier();

  u32x4_t ca[2][FM], cw[2][FN];
  uint32_t sc[FM + FN];
#pragma unroll
  for (int f = 0; f < FM + FN; ++f) read_code(0, 0, f, ca[0], cw[0]);
  read_scales(0, 0, true, sc);
  read_scales(0, 0, false, sc);

  constexpr int P = FM * FN, F = FM + FN;
  uint32_t hs[F];  // bytes 0 and 2: the lane half's blocks of the step's halves
  // quarter kk of a pair: its products, beside which the next quarter's fragments are read, in
  // the odd ones the next step's scales, and loads [l0, l1) of pair `to` are issued
  auto quarter = [&](auto which, int at, int kk_at, int to, int to_stage, int l0, int l1) __attribute__((always_inline)) {
    constexpr int kk = decltype(which)::value;
    const int reads = F + (kk & 1 ? 2 : 0);
    if constexpr ((kk & 1) == 0) {
#pragma unroll
      for (int f = 0; f < F; ++f) hs[f] = sc[f] >> (8 * h);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int j = p / FM, i = p % FM;
      if constexpr (kk & 1)
        acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(cw[1][j]), fp4_operand(ca[1][i]),
                                                                    acc[j][i], 4, 4, 2, (int)hs[FM + j], 2, (int)hs[i]);
      else
        acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(cw[0][j]), fp4_operand(ca[0][i]),
                                                                    acc[j][i], 4, 4, 0, (int)hs[FM + j], 0, (int)hs[i]);
      __builtin_amdgcn_sched_barrier(0);  // its wait for operands comes before the reads below
#pragma unroll
      for (int f = 0; f < reads; ++f) {
        if (f * (P * 3 / 4) / reads != p) continue;
        if (f < F) read_code(at, kk_at, f, ca[(kk & 1) ^ 1], cw[(kk & 1) ^ 1]);
        else read_scales(at, kk_at >> 1, f == F, sc);
      }
#pragma unroll
      for (int idx = l0; idx < l1; ++idx)
        if ((idx - l0) * P / (l1 - l0) == p) issue(to, to_stage, idx);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const int pairs = (a.groups + 1) / 2;
  int stage = 0;
  for (int ps = 0; ps < pairs; ++ps) {
    const int next = stage + 1 == kStages ? 0 : stage + 1, last = stage == 0 ? kStages - 1 : stage - 1;
    quarter(std::integral_constant<int, 0>(), stage, 1, ps - 1 + kStages, last, kEarly, T::Loads);
    quarter(std::integral_constant<int, 1>(), stage, 2, 0, 0, 0, 0);
    quarter(std::integral_constant<int, 2>(), stage, 3, 0, 0, 0, 0);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this stage's reads are done
    wait_loads<(kStages - 2) * T::Loads>();
    barrier();
    quarter(std::integral_constant<int, 3>(), next, 0, ps + kStages, stage, 0, kEarly);
    stage = next;
  }

  // ---- epilogue: 32 rows at a time through the wave's part of LDS, so that a store writes
  // whole row pieces. The loads past the last step are still writing zeros: wait first. ----
  wait_loads<0>();
  barrier();
  uint8_t* stg = smem + wave * (32 * T::RowBytes);
  constexpr int kChunks = 32 * FN / 8, kRowsPerStore = 64 / kChunks;
  const int64_t row0 = m0 + wm * FM * 32, col0 = n0 + wn * FN * 32;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(u32x2_t*)(stg + lr * T::RowBytes + (j * 32 + q * 8 + h * 4) * 2) =
            u32x2_t{pack_bf16(acc[j][i][q * 4], acc[j][i][q * 4 + 1]), pack_bf16(acc[j][i][q * 4 + 2], acc[j][i][q * 4 + 3])};
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int it = 0; it < 32 / kRowsPerStore; ++it) {
      const int r = it * kRowsPerStore + lane / kChunks, ch = lane % kChunks;
      const u32x4_t v = *(const u32x4_t*)(stg + r * T::RowBytes + ch * 16);
      const int64_t m = row0 + i * 32 + r, n = col0 + ch * 8;
      if (m < a.m && n < a.n) {
        uint16_t* dst = a.d + m * a.ldd + n;
        if (a.wide) {
          *(u32x4_t*)dst = v;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < a.n) dst[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
  }
}

// Workgroups go round-robin to the 8 XCDs: place b of count gets one contiguous range of
// them a XCD, numbered in bands of kBand M tiles, so that its L2 keeps the band's rows of A.
__device__ __forceinline__ int of_xcd(int b, int count) {
  const int per = count / 8, rem = count % 8, x = b & 7;
  return x * per + (x < rem ? x : rem) + (b >> 3);
}

struct Corner {
  int64_t m, n;
};

// of a tile, or of one of its parts: halves below each other, quarters two by two
__device__ __forceinline__ Corner corner(const MxGemmArgs& a, int tile, int part) {
  const int band = tile / (kBand * a.tiles_n);
  const int inside = tile - band * kBand * a.tiles_n;
  const int height = a.tiles_m - band * kBand < kBand ? a.tiles_m - band * kBand : kBand;
  return Corner{(int64_t)(band * kBand + inside % height) * kEdge + (part & 1) * (kEdge / 2),
                (int64_t)(inside / height) * kEdge + (part >> 1) * (kEdge / 2)};
}

// Whole tiles, and those of a last round that would leave half of the CUs idle or more as two
// or four parts each, a workgroup a part.
__global__ __launch_bounds__(64 * kWaves, 1) void mx_gemm_kernel(MxGemmArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int b = blockIdx.x;
  if (b < a.whole) {
    const Corner c = corner(a, of_xcd(b, a.whole), 0);
    run_tile<4, 4>(a, c.m, c.n, smem);
    return;
  }
  const Corner c = corner(a, a.whole + (b - a.whole) / a.parts, (b - a.whole) % a.parts);
  if (c.m >= a.m || c.n >= a.n) return;
  if (a.parts == 2) run_tile<2, 4>(a, c.m, c.n, smem);
  else run_tile<2, 2>(a, c.m, c.n, smem);
}

// Parts alone, where there is no whole tile: with registers for themselves they need no moves
// between the two register files, 23.1 -> 20.5 us for 512 x 5376 x 7168, 33.8 -> 30 for 1021.
template <int FM, int FN>
__global__ __launch_bounds__(64 * kWaves, 2) void mx_gemm_parts_kernel(MxGemmArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int p = of_xcd(blockIdx.x, a.tiles_m * a.tiles_n * a.parts);
  const Corner c = corner(a, p / a.parts, p % a.parts);
  if (c.m >= a.m || c.n >= a.n) return;
  run_tile<FM, FN>(a, c.m, c.n, smem);
}

// ---- few rows ------------------------------------------------------------------------------
// Up to 64 rows of A: the weight is read once and that is all there is to it. A workgroup
// takes 16 NT columns and its W waves split K; operands go from memory to registers
// (16x16x128: lane (r, u) has row r, block u of the step), a step ahead of their product. The
// waves' sums are joined in LDS in wave order. Every workgroup reads all of A, from L2: what
// A's registers cost beside the weight's decides NT (launch_mx_gemm).
// Measured, in a graph: 1 x 5376 x 14336 14.3 us (2.9 TB/s of weight, 2.7 us of it per
// launch). More steps ahead, or more waves, change nothing.
template <int MT, int NT, int W>
__global__ __launch_bounds__(64 * W, 2) void mx_gemm_thin_kernel(MxGemmArgs a) {
  __shared__ float red[W * MT * NT * 256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, u = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NT);
  const int krow = (int)(a.k >> 1), srow = a.groups * 512;
  const int rows_w = (int)(a.n - n0 < 16 * NT ? a.n - n0 : 16 * NT);
  __amdgpu_buffer_rsrc_t rA = __builtin_amdgcn_make_buffer_rsrc((void*)a.aq, 0, (int)a.m * krow, 0x00020000);
  __amdgpu_buffer_rsrc_t rW = __builtin_amdgcn_make_buffer_rsrc((void*)(a.wq + n0 * krow), 0, rows_w * krow, 0x00020000);
  __amdgpu_buffer_rsrc_t rSA = __builtin_amdgcn_make_buffer_rsrc((void*)a.as, 0, srow, 0x00020000);
  __amdgpu_buffer_rsrc_t rSW =
      __builtin_amdgcn_make_buffer_rsrc((void*)(a.ws + (n0 >> 7) * srow), 0, srow, 0x00020000);
  const int nrow = (int)(n0 & 127);  // the columns' rows in their 128-row scale tile
  auto scale_at = [&](int row) __attribute__((always_inline)) { return (row & 31) * 16 + (row >> 5) * 4; };

  f32x4_t acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // the waves share the K steps evenly, each a run of them
  struct Step {
    u32x4_t cw[NT], ca[MT];
    uint32_t sw[NT], sa[MT];
  };
  const int k_end = a.groups * (wave + 1) / W;
  auto load = [&](Step& x, int ks) __attribute__((always_inline)) {
    const int kb = ks * 64 + u * 16;
    const bool in = (kb < krow) & (ks < k_end);  // past K or the wave's run: codes 0, scales 0
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int row = j * 16 + r;
      x.cw[j] = __builtin_amdgcn_raw_buffer_load_b128(rW, in ? row * krow + kb : 0x7FFFFFF0, 0, 0);
      x.sw[j] = __builtin_amdgcn_raw_buffer_load_b32(rSW, in ? ks * 512 + scale_at(nrow + row) : 0x7FFFFFF0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int row = i * 16 + r;
      x.ca[i] = __builtin_amdgcn_raw_buffer_load_b128(rA, in ? row * krow + kb : 0x7FFFFFF0, 0, 0);
      x.sa[i] = __builtin_amdgcn_raw_buffer_load_b32(rSA, in ? ks * 512 + scale_at(row) : 0x7FFFFFF0, 0, 0);
    }
  };
  auto multiply = [&](const Step& x) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(x.cw[j]), fp4_operand(x.ca[i]), acc[j][i],
                                                                     4, 4, 0, (int)(x.sw[j] >> (8 * u)), 0,
                                                                     (int)(x.sa[i] >> (8 * u)));
  };
  Step x, y;
  int ks = a.groups * wave / W;
  load(x, ks);
  for (; ks < k_end; ks += 2) {
    load(y, ks + 1);
    __builtin_amdgcn_sched_barrier(0);
    multiply(x);
    __builtin_amdgcn_sched_barrier(0);
    load(x, ks + 2);
    __builtin_amdgcn_sched_barrier(0);
    multiply(y);
    __builtin_amdgcn_sched_barrier(0);
  }
  // lane (r, u) holds row m = r, columns 4u .. 4u + 3 of each 16 x 16 tile
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) *(f32x4_t*)(red + ((wave * NT + j) * MT + i) * 256 + lane * 4) = acc[j][i];
  __syncthreads();
  for (int e = threadIdx.x; e < MT * NT * 256; e += 64 * W) {
    // e: column within the workgroup's fastest, then row, so that stores run along D's rows
    const int col = e % (16 * NT), row = e / (16 * NT);
    const int at = ((col >> 4) * MT + (row >> 4)) * 256 + (((col & 15) >> 2) * 16 + (row & 15)) * 4 + (col & 3);
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) y += red[w * MT * NT * 256 + at];
    if (row < a.m && n0 + col < a.n) a.d[row * a.ldd + n0 + col] = (uint16_t)pack_bf16(y, 0.0f);
  }
}

constexpr int kLds = Shape<2, 4>::Lds;
static_assert(Shape<4, 4>::Lds <= kLds && Shape<2, 2>::Lds <= kLds && kLds <= 160 * 1024, "LDS");

// Whole rounds of 256 x 256 tiles, which need the fewest operand bytes a product; in a last
// round (or the only one) that fills at most half of the CUs, 128 x 256 halves, and 128 x 128
// quarters where even those fill at most half. Measured at N 5376, K 7168: 168 whole tiles
// take 57 us, 252 halves 38, 252 quarters 23. Parts are counted by tiles, also those without
// rows: of up to 128 rows half are empty and return at once (48 x 16128 x 5376: 126 of 252).
hipError_t launch_tiles(MxGemmArgs a, hipStream_t stream) {
  a.tiles_m = (int)((a.m + kEdge - 1) / kEdge);
  a.tiles_n = (int)((a.n + kEdge - 1) / kEdge);
  const int total = a.tiles_m * a.tiles_n, last = total % kCus;
  a.parts = last * 4 <= kCus ? 4 : last * 2 <= kCus ? 2 : 1;
  a.whole = a.parts == 1 ? total : total - last;
  const unsigned groups = (unsigned)(a.whole + (total - a.whole) * a.parts);
  if (a.whole > 0) mx_gemm_kernel<<<groups, 64 * kWaves, kLds, stream>>>(a);
  else if (a.parts == 2) mx_gemm_parts_kernel<2, 4><<<groups, 64 * kWaves, Shape<2, 4>::Lds, stream>>>(a);
  else mx_gemm_parts_kernel<2, 2><<<groups, 64 * kWaves, Shape<2, 2>::Lds, stream>>>(a);
  return hipGetLastError();
}

template <int MT, int NT>
hipError_t launch_thin_columns(const MxGemmArgs& a, hipStream_t stream) {
  constexpr int W = MT == 4 ? 4 : 8;
  mx_gemm_thin_kernel<MT, NT, W><<<(unsigned)((a.n + 16 * NT - 1) / (16 * NT)), 64 * W, 0, stream>>>(a);
  return hipGetLastError();
}

// As many columns a workgroup as still leave 160 workgroups (5 in 8 CUs): A is read once for
// each workgroup, so more columns save its bytes, but idle CUs cost more than they save.
// Measured for 1, 2 and 4 tiles: 1 x 5376 x 14336 17.5, 14.3, 23.3 us; 32 x 28672 x 5376 46,
// 33, 27 us; 64 x 5376 x 7168 26, 17.3, 23.5 us.
constexpr int64_t kThinGroups = 160;

template <int MT>
hipError_t launch_thin(const MxGemmArgs& a, hipStream_t stream) {
  if constexpr (MT < 4) {
    if (a.n >= kThinGroups * 64) return launch_thin_columns<MT, 4>(a, stream);
  }
  if (a.n >= kThinGroups * 32) return launch_thin_columns<MT, 2>(a, stream);
  return launch_thin_columns<MT, 1>(a, stream);
}

}  // namespace

hipError_t mx_gemm_setup() {
  constexpr auto kMost = hipFuncAttributeMaxDynamicSharedMemorySize;
  hipError_t e = hipFuncSetAttribute((const void*)mx_gemm_kernel, kMost, kLds);
  if (e == hipSuccess) e = hipFuncSetAttribute((const void*)mx_gemm_parts_kernel<2, 4>, kMost, Shape<2, 4>::Lds);
  if (e == hipSuccess) e = hipFuncSetAttribute((const void*)mx_gemm_parts_kernel<2, 2>, kMost, Shape<2, 2>::Lds);
  return e;
}

hipError_t launch_mx_gemm(const uint8_t* aq, const uint8_t* as, const uint8_t* wq, const uint8_t* ws, uint16_t* d,
                          int64_t ldd, int64_t m, int64_t n, int64_t k, hipStream_t stream) {
  MxGemmArgs a{aq, as, wq, ws, d, ldd, m, n, k, (int)((k / kMxBlock + 3) / 4), 0, 0, 0, 1,
               n % 8 == 0 && ldd % 8 == 0 && ((uintptr_t)d & 15u) == 0};
  // The thin form up to 32 rows, and up to 64 where a wide weight does not give the tiles
  // enough workgroups: 48 x 5376 x 7168 15.8 us, as tiles 18.0; 48 x 16128 x 5376 22.7 us, as
  // tiles 14.8; 32 x 5376 x 14336 21.6 us, as tiles 31.6.
  if (m <= 16) return launch_thin<1>(a, stream);
  if (m <= 32) return launch_thin<2>(a, stream);
  if (m <= 64 && n < kThinGroups * 64) return launch_thin<4>(a, stream);
  return launch_tiles(a, stream);
}

}  // namespace nvfp4
