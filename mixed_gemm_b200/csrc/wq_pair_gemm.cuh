// Pair-of-SMs tensor-core product shared by the INT8 product with token and
// channel scales and by the gated feed-forward (forward, input gradient,
// weight gradients):
//
//     D[m, n] = sum_k A[m, k] . B[n, k]        256 x BN per pair of CTAs
//
// A tile of D is computed by a cluster of two CTAs with
// tcgen05.mma.cta_group::2 (M = 256, N = BN): CTA r of the pair holds rows
// 128 r .. 128 r + 127 of A and of D, and BN / 2 of the BN rows of B.  At
// BN = 256 each SM therefore fetches 32 KB per 64-element (bf16; 128 for INT8)
// step of k for 512 cycles of tensor work, 64 bytes per cycle, where one CTA
// alone on a 128 x 256 tile would have to fetch 48 KB for the same 512
// cycles; shared memory filled from L2 is what bounds such a product first.
//
// An operand lies in memory either with k contiguous ("K-major", [rows, k]) or
// with its rows contiguous ("MN-major", [k, rows]); both are fetched by TMA in
// boxes of 128-byte rows with the 128-byte swizzle and described to the tensor
// core as they lie, so the gradients' products need no transposed copies.
// Elements past the tensors' ends are zero-filled by TMA, so any number of
// rows and any k is computed; the stores clip.
//
// Roles (384 threads per CTA): warp 0 issues the TMA loads of its
// CTA, completing on the first CTA's barrier; warp 1 of the first CTA issues
// the MMAs of the pair; warp 2 owns the tensor-memory allocation; warps 4..11
// read finished accumulators (two alternate, so the next tile's products run
// meanwhile), apply the epilogue and store through shared memory.  CTAs are
// persistent: pair p takes tiles p, p + pairs, ...  Every wait on a barrier has
// an iteration limit; one that runs out sets the error word and winds down.
//
// Bound by the tensor pipe at the clock that the power limit leaves: INT8 4096 x 8192 x
// 8192 192 us (2.9 POPS; 4.1 on zeros), both gated projections 4096 x 24576 x 4096 with
// their epilogue 620 us (1.33 PFLOP/s; 2.1 on zeros), dx of 4096 x 4096 over 24576 519
// us, both dW 565 to 620.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "wq_act_fn.cuh"
#include "wq_ff.cuh"
#include "wq_internal.cuh"
#include "wq_tc.cuh"

namespace wq {

// What the epilogue makes of the sums.
enum PairEpi {
  EPI_I8_BF16 = 0,  // s32 sums x token scale x channel scale (+ bias) -> bf16
  EPI_I8_F32 = 1,   // the same, fp32 out
  EPI_GATED = 2,    // columns [gate | up]: act(gate + bg) (up + bu) -> bf16, both
                    // pre-activations too where they are kept
  EPI_DX = 3,       // bf16; the sum runs over two pairs of operands
  EPI_DW = 4        // bf16; two A operands, each with its own output
};

// Place of tile t among tm x tn tiles: bands of eight rows of tiles, so that the pairs at
// work share a few rows of A and of B in L2.
__host__ __device__ inline void pair_tile(int t, int tm, int tn, int* mt, int* nt) {
  const int band = t / (8 * tn), in = t - band * 8 * tn;
  const int rows = tm - band * 8 < 8 ? tm - band * 8 : 8;
  *mt = band * 8 + in % rows;
  *nt = in / rows;
}

struct PairMaps {
  CUtensorMap a[2], b[2], out[3];
};

struct PairParams {
  int M, N;          // rows and columns of one output (gated: columns of h)
  int KT, kt_split;  // ring slots of k in all; those of the first pair of operands (EPI_DX)
  int tiles_m, tiles_n, tiles;  // tiles_m: of one output
  // EPI_DX, EPI_DW: tiles from `whole` on come in `splits` parts of k, each an fp32 tile of
  // partial sums in out[2], to be added by another kernel
  int whole, splits;
  int tma_out;       // outputs are stored by TMA (rows a multiple of 16 bytes)
  int save;
  const float* sx;
  const float* sw;
  const uint16_t* bias0;
  const uint16_t* bias1;
  void* out[3];
#ifdef WQ_FAULT_TEST
  int fault;  // test build only: finished accumulators are not announced, so the
              // epilogue's bounded wait runs out; no copy or product is altered
#endif
};

// the kernels' error word (wq_device_error bits 512 producer, 1024 the ends of
// copies and products in flight, 2048 MMA issuer, 4096 epilogue, 8192 misaligned shared memory)
__device__ unsigned g_wq_pair_error;

constexpr int kPairThreads = 384;
constexpr int kEpiWarps = 8;
constexpr uint32_t kPairStageOut = 4096;  // one warp's 32 rows x 128 bytes

template <int EPI, int BN>
struct PairCfg {
  static constexpr bool kI8 = EPI == EPI_I8_BF16 || EPI == EPI_I8_F32;
  static constexpr bool kDX = EPI == EPI_DX;
  static constexpr bool kDW = EPI == EPI_DW;
  static constexpr bool kF32 = EPI == EPI_I8_F32;
  static constexpr bool kAmn = kDW;
  static constexpr bool kBmn = kDX || kDW;
  static constexpr int KS = kI8 ? 128 : 64;  // k per block: 128 bytes of a K-major row
  // Blocks of k per ring slot.  A slot costs the issuing warp about 400 cycles of
  // waits, MMAs and commits whatever its size; one block at BN = 256 keeps the tensor
  // cores busy for 512, at 128 for 256 and at 64 for 128, so the narrow tiles
  // take two.
  static constexpr int kBlocks = BN == 256 ? 1 : 2;
  static constexpr uint32_t kAbytes = 128 * 128;
  static constexpr uint32_t kBbytes = (BN / 2) * 128;
  static constexpr uint32_t kBlock = kAbytes + kBbytes;
  static constexpr uint32_t kSlot = kBlocks * kBlock;
  // output staging: a buffer an epilogue warp; column data (scales, biases): 2 x 32 floats
  static constexpr uint32_t kStaging = kEpiWarps * kPairStageOut;
  static constexpr uint32_t kColumns = kEpiWarps * 64 * 4;
  static constexpr uint32_t kFixed = kStaging + kColumns + 256;
  static constexpr int kFit = (int)((227u * 1024u - kFixed) / kSlot);
  static constexpr int ST = kFit > 8 ? 8 : kFit;
  static constexpr uint32_t kSmem = kFixed + ST * kSlot;
  static constexpr uint32_t kTmemCols = 2 * BN;
  // columns of the output that one tile covers, and columns per stored chunk
  static constexpr int kTileN = EPI == EPI_GATED ? BN / 2 : BN;
  static constexpr int kChunk = kF32 ? 32 : 64;
  static_assert(ST >= 3, "ring too short");
  static_assert(kTileN % kChunk == 0 && kTileN / kChunk >= 1, "a tile is whole chunks");
  static_assert(!kBmn || BN >= 128, "an MN-major box is 64 rows");
};

// ACT: the gated epilogue's activation (others: 0).  A constant, so that only its own
// code is fetched: with all three behind a branch a 2048 x 2048 gated product of 64
// tokens took 18.7 us.
template <int EPI, int BN, int ACT>
__global__ void __launch_bounds__(kPairThreads, 1)
    pair_gemm_kernel(const __grid_constant__ PairMaps maps, const PairParams p) {
  unsigned* const err = &g_wq_pair_error;
  using C = PairCfg<EPI, BN>;
  constexpr int ST = C::ST;
  // the pair's CTAs run one kernel with one shared-memory layout, so an offset
  // means the same place in both
  extern __shared__ __align__(1024) uint8_t smem[];
  if (tc::smem_u32(smem) & 1023u) {  // the operand tiles' swizzle needs the alignment
    atomicOr(err, 8192u);
    return;
  }
  uint8_t* staging = smem + ST * C::kSlot;
  float* columns = (float*)(staging + C::kStaging);
  uint64_t* bars = (uint64_t*)((uint8_t*)columns + C::kColumns);
  uint32_t* tmem_slot = (uint32_t*)(bars + 2 * ST + 5);
  volatile int* abort = (volatile int*)(tmem_slot + 1);
  auto full_bar = [&](int s) { return tc::smem_u32(bars + s); };
  auto empty_bar = [&](int s) { return tc::smem_u32(bars + ST + s); };
  auto tfull_bar = [&](int b) { return tc::smem_u32(bars + 2 * ST + b); };
  auto tempty_bar = [&](int b) { return tc::smem_u32(bars + 2 * ST + 2 + b); };
  const uint32_t drain_bar = tc::smem_u32(bars + 2 * ST + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)tc::cluster_rank();
  const int pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      tc::mbar_init(full_bar(s), 1);   // the first CTA's producer; both CTAs' bytes
      tc::mbar_init(empty_bar(s), 1);  // the MMA issuer's commit
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(tfull_bar(b), 1);
      tc::mbar_init(tempty_bar(b), 2 * kEpiWarps);  // the epilogue warps of both CTAs
    }
    tc::mbar_init(drain_bar, 1);
    *abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 2) tc::tmem_alloc2(tc::smem_u32(tmem_slot), C::kTmemCols);
  if (warp == 3 && lane == 0) {
    tc::prefetch_map(&maps.a[0]);
    tc::prefetch_map(&maps.b[EPI == EPI_GATED ? rank : 0]);
    if (p.tma_out) tc::prefetch_map(&maps.out[0]);
  }
  tc::fence_before();
  tc::cluster_sync();
  tc::fence_after();
  // Launched as a programmatic dependent: all of the above ran beside the end of the
  // kernel before, nothing of it touches its data.  The next kernel may start its
  // own once the kernel before is complete.
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t tmem = *tmem_slot;

  struct Tile {
    int m0, n0, sel, kt0, kt1;
    int part;  // which tile of partial sums, or -1: the output itself
  };
  const int tm_all = C::kDW ? 2 * p.tiles_m : p.tiles_m;
  auto tile_at = [&](int t) -> Tile {
    Tile u;
    u.kt0 = 0;
    u.kt1 = p.KT;
    u.part = -1;
    if (C::kBmn && t >= p.whole) {  // the parts of a tile side by side
      u.part = t - p.whole;
      const int split = u.part % p.splits;
      t = p.whole + u.part / p.splits;
      u.kt0 = (int)((int64_t)p.KT * split / p.splits);
      u.kt1 = (int)((int64_t)p.KT * (split + 1) / p.splits);
    }
    int mt, nt;
    pair_tile(t, tm_all, p.tiles_n, &mt, &nt);
    u.sel = C::kDW && mt >= p.tiles_m ? 1 : 0;
    if (u.sel) mt -= p.tiles_m;
    u.m0 = mt * 256;
    u.n0 = nt * C::kTileN;
    return u;
  };

  // Producer and MMA issuer run as whole, converged warps whose elected lane issues:
  // addresses and descriptors then stay in uniform registers, which the TMA and
  // tcgen05 instructions take.
  if (warp == 0) {
    // -------------------------------------------------------------- producer
    int s = 0;
    uint32_t ph = 1;  // of the slot's release: the first round finds it free
    int use = 0;
    bool run = true;
    for (int t = pair; t < p.tiles && run; t += pairs) {
      const Tile u = tile_at(t);
      const int am = u.m0 + rank * 128;
      const int bn = EPI == EPI_GATED ? u.n0 : u.n0 + rank * (BN / 2);
      for (int kt = u.kt0; kt < u.kt1; ++kt, ++use) {
        if (use >= ST && !tc::warp_wait(empty_bar(s), ph, abort, err, 512u)) {
          run = false;
          break;
        }
        const int seg = C::kDX && kt >= p.kt_split ? 1 : 0;
        const int k0 = (seg ? kt - p.kt_split : kt) * (C::kBlocks * C::KS);
        const CUtensorMap* ma = &maps.a[C::kDX ? seg : u.sel];
        const CUtensorMap* mb = &maps.b[EPI == EPI_GATED ? rank : seg];
        const uint32_t slot = tc::smem_u32(smem + s * C::kSlot);
        const uint32_t bar = tc::map_to_rank(full_bar(s), 0);
        if (tc::elect()) {
          if (rank == 0) tc::mbar_expect_tx(full_bar(s), 2 * C::kSlot);
          // (a last slot's second block may start past the end of k: zeros)
#pragma unroll
          for (int h = 0; h < C::kBlocks; ++h) {
            const int k = k0 + h * C::KS;
            const uint32_t da = slot + h * C::kBlock, db = da + C::kAbytes;
            if constexpr (C::kAmn) {
              tc::tma_load2(da, ma, am, k, bar);
              tc::tma_load2(da + 8192, ma, am + 64, k, bar);
            } else {
              tc::tma_load2(da, ma, k, am, bar);
            }
            if constexpr (C::kBmn) {
#pragma unroll
              for (int j = 0; j < BN / 128; ++j)
                tc::tma_load2(db + j * 8192, mb, bn + 64 * j, k, bar);
            } else {
              tc::tma_load2(db, mb, k, bn, bar);
            }
          }
        }
        __syncwarp();
        if (++s == ST) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // before this CTA may leave: no load into it in flight (the first CTA's
    // barriers count both CTAs' bytes), no commit on its way to its barriers
    for (int v = use < ST ? 0 : use - ST; v < use; ++v) {
      if (rank == 0)
        tc::warp_wait(full_bar(v % ST), (uint32_t)(v / ST) & 1u, abort, err, 1024u, false);
      if (run) tc::warp_wait(empty_bar(v % ST), (uint32_t)(v / ST) & 1u, abort, err, 1024u);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc = ((C::kI8 ? 2u : 1u) << 4) | (1u << 7) | (1u << 10) |
                                 ((C::kAmn ? 1u : 0u) << 15) | ((C::kBmn ? 1u : 0u) << 16) |
                                 ((uint32_t)(BN >> 3) << 17) | ((256u >> 4) << 24);
      // descriptors of slot 0; a slot and a step of 32 bytes of k (K-major) or of
      // 16 rows of 128 bytes (MN-major) are adds to the address field
      const uint32_t base = tc::smem_u32(smem);
      const uint64_t a0 = C::kAmn ? tc::desc_mn(base) : tc::desc_k(base);
      const uint64_t b0 = C::kBmn ? tc::desc_mn(base + C::kAbytes) : tc::desc_k(base + C::kAbytes);
      constexpr uint32_t sa = C::kAmn ? 128 : 2, sb = C::kBmn ? 128 : 2;
      int s = 0, i = 0;
      uint32_t ph = 0;
      bool ok = true, ready = false;
      for (int t = pair; t < p.tiles && ok; t += pairs, ++i) {
        const int b = i & 1;
        if (i >= 2 &&
            !tc::warp_wait(tempty_bar(b), (uint32_t)((i >> 1) - 1) & 1u, abort, err, 2048u)) {
          ok = false;
          break;
        }
        tc::fence_after();
        const uint32_t d = tmem + (uint32_t)(b * BN);
        const Tile u = tile_at(t);
        for (int kt = u.kt0; kt < u.kt1; ++kt) {
          if (!ready && !tc::warp_wait(full_bar(s), ph, abort, err, 2048u)) {
            ok = false;
            break;
          }
          tc::fence_after();
          const uint32_t at = (uint32_t)s * (C::kSlot >> 4);
          if (++s == ST) {
            s = 0;
            ph ^= 1u;
          }
          // look at the next slot's barrier now, so that the answer comes while this
          // slot's MMAs are issued
          const bool seen = tc::mbar_test(full_bar(s), ph);
          if (tc::elect()) {
#pragma unroll
            for (int h = 0; h < C::kBlocks; ++h)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc::mma2<C::kI8>(d, a0 + at + h * (C::kBlock >> 4) + kk * sa,
                                 b0 + at + h * (C::kBlock >> 4) + kk * sb, idesc,
                                 ((kt - u.kt0) | h | kk) != 0);
            tc::commit2(empty_bar(s == 0 ? ST - 1 : s - 1));
          }
          ready = __all_sync(0xffffffffu, seen);
        }
        bool announce = ok;
#ifdef WQ_FAULT_TEST
        announce = ok && !p.fault;
#endif
        if (announce && tc::elect()) tc::commit2(tfull_bar(b));
        __syncwarp();
      }
      if (!ok) {  // the MMAs issued end before the memory goes away
        if (tc::elect()) tc::commit1of2(drain_bar);
        __syncwarp();
        tc::warp_wait(drain_bar, 0u, abort, err, 1024u, false);
      }
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    // warp w reads the 32 accumulator rows of its quadrant, every second chunk of columns
    const int ew = warp & 3, half = (warp - 4) >> 2;
    uint8_t* stage = staging + (warp - 4) * kPairStageOut;
    float* col0 = columns + (warp - 4) * 64;
    float* col1 = col0 + 32;
    int i = 0;
    // one chunk's 32 rows, staged by this warp, to out[which]
    auto store_chunk = [&](auto f32, int which, int row0, int n0) {
      uint8_t* src = stage;
      constexpr int E = decltype(f32)::value ? 4 : 2;
      if (p.tma_out) {
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::tma_store(&maps.out[which], n0, row0, tc::smem_u32(src));
          tc::bulk_commit();
        }
      } else {
        // rows that are no multiple of 16 bytes: element by element, a row's 128 bytes by
        // the lanes side by side, eight rows on their way at once
        __syncwarp();
        const int cols = min(128 / E, p.N - n0);
        constexpr int kPer = 4 / E;  // elements of a row that a lane stores
#pragma unroll 1
        for (int r0 = 0; r0 < 32; r0 += 8) {
          uint32_t v[8][kPer];
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              const int r = r0 + i, c = lane + 32 * e;
              const uint8_t* at = src + r * 128 + ((((c * E) >> 4) ^ (r & 7)) << 4) + ((c * E) & 15);
              v[i][e] = E == 4 ? *(const uint32_t*)at : *(const uint16_t*)at;
            }
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              const int r = row0 + r0 + i, c = lane + 32 * e;
              const int64_t o = (int64_t)r * p.N + n0 + c;
              if (r < p.M && c < cols) {
                if constexpr (E == 4)
                  ((uint32_t*)p.out[which])[o] = v[i][e];
                else
                  ((uint16_t*)p.out[which])[o] = (uint16_t)v[i][e];
              }
            }
        }
        __syncwarp();
      }
    };
    // the staging buffer is free
    auto next_buffer = [&]() {
      if (p.tma_out && lane == 0) tc::bulk_wait_read_all();
      __syncwarp();
    };
    // 16 bytes (chunk j of the row) of this lane's row of the staging buffer
    auto stage16 = [&](int j, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
      *(uint4*)(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
          make_uint4(a, b, c, d);
    };
    for (int t = pair; t < p.tiles; t += pairs, ++i) {
      const Tile u = tile_at(t);
      const int b = i & 1;
      const int row0 = u.m0 + rank * 128 + ew * 32;
      float sx = 0.f;
      if constexpr (C::kI8)
        if (row0 + lane < p.M) sx = __ldg(p.sx + row0 + lane);
      // one answer for the warp: the reads below are of whole warps
      __syncwarp();
      if (!tc::warp_wait(tfull_bar(b), (uint32_t)(i >> 1) & 1u, abort, err, 4096u)) break;
      tc::fence_after();
      const uint32_t acc = tmem + (uint32_t)(b * BN) + ((uint32_t)(ew * 32) << 16);
      // 32 columns' data, broadcast to the lanes from shared memory
      auto column_data = [&](int n) {
        if constexpr (C::kI8 || EPI == EPI_GATED) {
          __syncwarp();
          const bool in = n + lane < p.N;
          if constexpr (C::kI8) {
            col0[lane] = in ? __ldg(p.sw + n + lane) : 0.f;
            col1[lane] = in && p.bias0 ? bf16_bits_to_f32(__ldg(p.bias0 + n + lane)) : 0.f;
          } else {
            col0[lane] = in && p.bias0 ? bf16_bits_to_f32(__ldg(p.bias0 + n + lane)) : 0.f;
            col1[lane] = in && p.bias1 ? bf16_bits_to_f32(__ldg(p.bias1 + n + lane)) : 0.f;
          }
          __syncwarp();
        }
      };
      // one chunk of 128 bytes a row (64 bf16 or 32 fp32 columns) from column c of the
      // accumulator to (row, column) of out[which]
      auto chunk = [&](auto f32, int c, int which, int row, int col) {
        constexpr bool F32 = decltype(f32)::value;
        constexpr int CH = F32 ? 32 : 64;
        const int n0 = u.n0 + c;
        // all of the chunk is read and computed while the last store still reads the
        // buffer
        uint32_t v[CH / 16][16];
#pragma unroll
        for (int q = 0; q < CH / 16; ++q) tc::tmem_ld16(acc + c + 16 * q, v[q]);
#pragma unroll
        for (int q = 0; q < CH / 16; ++q) {
          if ((q & 1) == 0) column_data(n0 + 16 * q);
          tc::tmem_wait_ld(v[q]);
          if constexpr (C::kI8) {
            // one rounding of the exact sum to fp32, then two products and
            // the bias in fp32
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 w4 = *(const float4*)(col0 + (q & 1) * 16 + j);
              const float4 b4 = *(const float4*)(col1 + (q & 1) * 16 + j);
              v[q][j] = __float_as_uint((float)(int)v[q][j] * sx * w4.x + b4.x);
              v[q][j + 1] = __float_as_uint((float)(int)v[q][j + 1] * sx * w4.y + b4.y);
              v[q][j + 2] = __float_as_uint((float)(int)v[q][j + 2] * sx * w4.z + b4.z);
              v[q][j + 3] = __float_as_uint((float)(int)v[q][j + 3] * sx * w4.w + b4.w);
            }
          }
          if constexpr (!F32)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              v[q][j] = pack_bf16(__uint_as_float(v[q][2 * j]), __uint_as_float(v[q][2 * j + 1]));
        }
        next_buffer();
#pragma unroll
        for (int q = 0; q < CH / 16; ++q)
#pragma unroll
          for (int j = 0; j < (F32 ? 16 : 8); j += 4)
            stage16((q * (F32 ? 16 : 8) + j) / 4, v[q][j], v[q][j + 1], v[q][j + 2], v[q][j + 3]);
        store_chunk(f32, which, row, col);
      };
      if (row0 < p.M) {
        if (C::kBmn && u.part >= 0) {
#pragma unroll 1
          for (int c = half * 32; c < BN && u.n0 + c < p.N; c += 64)
            chunk(std::true_type{}, c, 2, u.part * 256 + rank * 128 + ew * 32, c);
        } else {
#pragma unroll 1
          for (int c = half * C::kChunk; c < C::kTileN; c += 2 * C::kChunk) {
            const int n0 = u.n0 + c;
            if (n0 >= p.N) break;
            if constexpr (EPI == EPI_GATED) {
              // h, then (kept for the backward pass) the pre-activations
              const int outs = p.save ? 3 : 1;
#pragma unroll 1
              for (int o = 0; o < outs; ++o) {
#pragma unroll 1
                for (int q = 0; q < 64; q += 16) {
                  if ((q & 31) == 0) column_data(n0 + q);
                  uint32_t g[16], w[16];
                  tc::tmem_ld16(acc + c + q, g);
                  tc::tmem_ld16(acc + BN / 2 + c + q, w);
                  tc::tmem_wait_ld(g);
                  tc::tmem_wait_ld(w);
                  uint32_t h[8];
#pragma unroll
                  for (int j = 0; j < 16; j += 4) {
                    const float4 b0 = *(const float4*)(col0 + (q & 16) + j);
                    const float4 b1 = *(const float4*)(col1 + (q & 16) + j);
                    const float ba[4] = {b0.x, b0.y, b0.z, b0.w}, bb[4] = {b1.x, b1.y, b1.z, b1.w};
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                      const float gg = __uint_as_float(g[j + e]) + ba[e];
                      const float uu = __uint_as_float(w[j + e]) + bb[e];
                      v[e] = o == 0 ? act_value(ACT, gg) * uu : o == 1 ? gg : uu;
                    }
                    h[j / 2] = pack_bf16(v[0], v[1]);
                    h[j / 2 + 1] = pack_bf16(v[2], v[3]);
                  }
                  if (q == 0) next_buffer();
                  stage16(q / 8, h[0], h[1], h[2], h[3]);
                  stage16(q / 8 + 1, h[4], h[5], h[6], h[7]);
                }
                store_chunk(std::false_type{}, o, row0, n0);
              }
            } else {
              chunk(std::integral_constant<bool, C::kF32>{}, c, u.sel, row0, n0);
            }
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_rank0(tempty_bar(b));
    }
    if (p.tma_out && lane == 0) tc::bulk_wait_read_all();
  }
  __syncwarp();
  tc::fence_before();
  tc::cluster_sync();
  if (warp == 2) {
    tc::fence_after();
    tc::tmem_dealloc2(tmem, C::kTmemCols);
  }
}

}  // namespace wq
