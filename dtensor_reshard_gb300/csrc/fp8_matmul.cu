// fp8_matmul.cu -- reshard_fp8_matmul: the product of e4m3 matrices with a float32
// scale for each block of 128, dense or one weight matrix for each expert.
//
// The scales change every 128 steps of k, so no tensor-core accumulator can run through
// them: the matrix instructions of one block of 128 write a fresh accumulator in tensor
// memory, and the threads that own its rows add scale * accumulator to float32 sums in
// registers while the next block is multiplied into another accumulator.
//
// Two kernels, which differ in what lies in the accumulator's 128 lanes (its rows):
//   wide    128 tokens x 256 features a CTA: tokens in the lanes, so a thread has one token
//           scale and one weight scale a block;
//   narrow  128 features x NT tokens a CTA: weights in the lanes, so that few tokens
//           (MMA N down to 16) still use whole instructions; bound by reading w.
#include <cudaTypedefs.h>

#include <atomic>

#include "operators.cuh"
#include "tensor_core.cuh"

namespace rs {
namespace {

using namespace op;
using staging::mbar_arrive_expect;
using staging::mbar_init;

constexpr int kBlock = 128;           // values of k that share a scale, bytes of a tile row
constexpr int kRows = 128;            // rows of a loaded tile
constexpr int kTileBytes = kRows * kBlock;
constexpr int kMostSplit = 8;         // CTAs of a cluster that share the blocks of k

// Codes for the device status word (staging.cuh has 1 to 4).
enum : unsigned int {
  kStatusLoadWait = 5,    // the loading warp gave up waiting for a free stage
  kStatusMatrixWait = 6,  // the matrix warp gave up waiting for data or an accumulator
  kStatusSumWait = 7      // a summing warp gave up waiting for an accumulator
};

struct MatmulArgs {
  const float *xs, *ws;
  int64_t ldxs, ldws;
  const int32_t* offsets;
  int32_t nexperts, tokens, n, blocks;  // blocks of k
  int32_t ntiles, col_blocks;           // tiles and scale blocks along n
  void* y;
  int64_t ldy;
  uint32_t* status;
  int32_t aligned_y;  // every row of y starts on 32 or 16 bytes, or 0
};

// Each expert's first row and first tile, in shared memory: start[e], tiles[e] for
// e <= nexperts.  `rows` rows make a tile along the tokens, ntiles tiles lie along n.
struct ExpertTable {
  int *start, *tiles;
  __device__ ExpertTable(char* smem, int nexperts)
      : start(reinterpret_cast<int*>(smem)), tiles(start + nexperts + 1) {}
  __host__ __device__ static constexpr size_t bytes(int64_t nexperts) { return size_t(8 * (nexperts + 1)); }

  __device__ void build(const MatmulArgs& a, int rows) {
    const int lane = threadIdx.x & 31;
    if (a.offsets == nullptr) {
      if (threadIdx.x == 0) {
        start[0] = tiles[0] = 0;
        start[1] = a.tokens;
        tiles[1] = (a.tokens + rows - 1) / rows * a.ntiles;
      }
      return;
    }
    for (int i = threadIdx.x; i <= a.nexperts; i += blockDim.x)
      start[i] = min(max(a.offsets[i], 0), a.tokens);
    __syncthreads();
    if (threadIdx.x >= 32) return;
    int most = 0, sum = 0;  // an offset below an earlier one counts as that one
    for (int base = 0; base <= a.nexperts; base += 32) {
      const int i = base + lane;
      int v = max(i <= a.nexperts ? start[i] : 0, most);
      for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = max(v, w);
      }
      if (i <= a.nexperts) start[i] = v;
      most = __shfl_sync(0xffffffffu, v, 31);
    }
    __syncwarp();
    for (int base = 0; base < a.nexperts; base += 32) {
      const int i = base + lane;
      int v = i < a.nexperts ? (start[i + 1] - start[i] + rows - 1) / rows * a.ntiles : 0;
      for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
      }
      if (i < a.nexperts) tiles[i + 1] = sum + v;
      sum += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) tiles[0] = 0;
  }
};

// One tile: rows [row, end) of expert e (at most a tile's), features from n0.
struct Tile {
  int e, row, end, n0;
  __device__ Tile() : e(0), row(0), end(0), n0(0) {}
  __device__ Tile(const ExpertTable& t, int nexperts, int index, int rows, int cols) {
    int lo = 0, hi = nexperts - 1;  // the last expert whose first tile is not after index
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.tiles[mid] <= index) lo = mid;
      else hi = mid - 1;
    }
    e = lo;
    const int per_col = (t.start[e + 1] - t.start[e] + rows - 1) / rows;
    const int i = index - t.tiles[e];
    row = t.start[e] + i % per_col * rows;
    end = t.start[e + 1];
    n0 = i / per_col * cols;
  }
};

constexpr size_t kTableMost = 8 * (RESHARD_MAX_EXPERTS + 1);  // ExpertTable::bytes

// After a wait ran out: time for this thread's copies and matrix instructions to land
// before shared and tensor memory are given back.
__device__ __noinline__ void give_up(uint32_t* status, uint32_t code) {
  atomicExch(status, code);
  for (int i = 0; i < 64; ++i) __nanosleep(100000);
}

// ------------------------------------------------------------------------------- wide
// Twelve warps a CTA, which takes 128 tokens x 256 features, loads both for every block (a 48
// KiB stage), and sums with two warps a lane quarter, 128 columns each.  Every CTA loads its own
// tiles: the tiles of a launch go along the tokens first, so that CTAs at work at a time read
// the same weights from L2.
// What bounds it is the accumulators' way out of tensor memory, which the matrix instructions need
// too, and into the sums: 8192 x 14336 x 4096 to bf16 takes 420 to 455 us, by the clock that the
// power cap leaves (2.1 to 2.3 PFLOP/s), 307 us with all loads of accumulators but an eighth of the
// additions; the tensor pipe is active 48% of the time, and L2 gives 12.6 TB/s.  Two accumulators of 256
// columns fill the 512: as four of 128 columns, with 16 summing warps, with tensor-memory loads
// of 32 columns or with scalar sums it was slower by 4 to 70%.
// 16384 tokens over 16 experts of [2048, 7168]: 255 us (1.9 PFLOP/s).
constexpr int kWideStages = 4;  // 2 where the expert table needs the room
constexpr int kWideStageBytes = 3 * kTileBytes;
constexpr int kWideCols = 256;
constexpr int kWideSumWarps = 8;
constexpr int kWideWarpCols = kWideCols / (kWideSumWarps / 4);
constexpr int kWideThreads = 32 * (kWideSumWarps + 4);
constexpr int kOutRow = 64;              // bytes of an output row staged at a time
constexpr int kOutPitch = kOutRow + 16;  // no bank conflicts where rows are written
constexpr int kOutBytes = 32 * kOutPitch;

// A summing warp fetches the scales of its 32 rows for 8 blocks at a time, a sector a
// row, and keeps the products of both scales in shared memory (one word a lane and block:
// reading xs where it lies would touch 32 lines for each block).
constexpr int kScaleBlocks = 8;
constexpr int kScalePitch = kScaleBlocks + 1;

// Shares of the register file, a warp: 8 * 224 + 4 * 56 = 12 * 168 at launch.
constexpr int kWideSumRegisters = 224, kWideOtherRegisters = 56;

// What lies before the stages in shared memory.
struct WideSmem {
  alignas(16) unsigned char out[kWideSumWarps][kOutBytes];
  float scales[kWideSumWarps][32 * kScalePitch];
  uint64_t full[kWideStages], empty[kWideStages], sum_full[2], sum_empty[2];
  uint32_t tmem;
};
// Offset of the stages: behind WideSmem and the table, on a swizzle atom.
__host__ __device__ constexpr size_t wide_stages_at(size_t table_bytes) {
  return (sizeof(WideSmem) + table_bytes + 1023) / 1024 * 1024;
}
static_assert(wide_stages_at(kTableMost) + 2 * kWideStageBytes <= kSmemMost, "shared memory");

// For fewer tokens than fill the GPU that way, such a tile a cluster, of which each CTA
// takes a share of the blocks of k; the sums of 16 columns at a time go to the CTA that
// adds them up, in rank order, through distributed shared memory (in the place of the
// stages).  64 x 7168 x 7168 takes 17.3 us, 128 tokens 20 us, by five CTAs a tile, against
// 25 us with 64-token tiles; 513 x 2688 x 7168 by two 26 us.
constexpr int kSplitChunk = 16;  // columns
constexpr int kSplitChunkBytes = kRows * kSplitChunk * 4;
// Chunks that a CTA receives at most, from all CTAs of a split.
__host__ __device__ constexpr int split_chunks(int split) {
  return (kWideCols / kSplitChunk + split - 1) / split * split;
}

template <typename Y>
__global__ void __launch_bounds__(kWideThreads, 1)
    wide_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                const __grid_constant__ MatmulArgs a, const int stages) {
  extern __shared__ __align__(1024) unsigned char dynamic[];
  WideSmem& sm = *reinterpret_cast<WideSmem*>(dynamic);
  ExpertTable table(reinterpret_cast<char*>(dynamic + sizeof(WideSmem)), a.nexperts);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_rank();
  uint32_t ctas;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const int unit = blockIdx.x / ctas, units = gridDim.x / ctas;
  const int b0 = int(int64_t(a.blocks) * rank / ctas);
  const int b1 = int(int64_t(a.blocks) * (rank + 1) / ctas);
  const uint32_t data =
      staging::smem_addr(dynamic) + uint32_t(wide_stages_at(ExpertTable::bytes(a.nexperts)));

  if (threadIdx.x == 0) {
    tc::prefetch_map(&map_x);
    tc::prefetch_map(&map_w);
    for (int i = 0; i < stages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.sum_full[i], 1);
      mbar_init(&sm.sum_empty[i], kWideSumWarps);
    }
    tc::fence_barrier_init();
  }
  if (warp == kWideSumWarps + 1) tc::tmem_alloc(&sm.tmem, 512);
  table.build(a, kRows);
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem;
  const int total = table.tiles[a.nexperts];

  if (warp == kWideSumWarps) {  // loads
    tc::registers_down<kWideOtherRegisters>();
    uint32_t stage = 0, parity = 1;
    bool ok = true;
    for (int t = unit; ok && t < total; t += units) {
      const Tile tile(table, a.nexperts, t, kRows, kWideCols);
      for (int b = b0; b < b1; ++b) {
        if (!(ok = tc::warp_wait(&sm.empty[stage], parity))) break;
        if (lane == 0) {
          mbar_arrive_expect(&sm.full[stage], kWideStageBytes);
          const uint32_t bar = staging::smem_addr(&sm.full[stage]);
          const uint32_t dst = data + stage * kWideStageBytes;
          tc::load_box(dst, &map_x, bar, b * kBlock, tile.row, 0);
          tc::load_box(dst + kTileBytes, &map_w, bar, b * kBlock, tile.n0, tile.e);
          tc::load_box(dst + 2 * kTileBytes, &map_w, bar, b * kBlock, tile.n0 + kRows, tile.e);
        }
        __syncwarp();
        if (++stage == uint32_t(stages)) stage = 0, parity ^= 1;
      }
    }
    // every matrix instruction has let go of its stage before this CTA may end
    for (int i = 0; ok && i < stages; ++i) {
      ok = tc::warp_wait(&sm.empty[stage], parity);
      if (++stage == uint32_t(stages)) stage = 0, parity ^= 1;
    }
    if (!ok && lane == 0) give_up(a.status, kStatusLoadWait);
  } else if (warp > kWideSumWarps) {
    tc::registers_down<kWideOtherRegisters>();
    if (warp <= kWideSumWarps + 2) {  // matrix instructions
      constexpr uint32_t instruction = tc::e4m3_instruction(kRows, kWideCols);
      // This warp's accumulator, for every other block; the stages are two or four, so that
      // each is one warp's too (a barrier's phases are told apart by parity, which only holds
      // for a warp that sees all of them).
      const uint32_t buf = warp - (kWideSumWarps + 1);
      const int count = unit < total ? ((total - 1 - unit) / units + 1) * (b1 - b0) : 0;
      uint32_t stage = buf, parity = 0, buf_parity = 1;
      bool ok = true;
      for (int i = buf; i < count; i += 2) {
        const uint32_t src = data + stage * kWideStageBytes;
        const uint64_t dx = tc::tile_desc(src), dw = tc::tile_desc(src + kTileBytes);
        // the accumulator last: it is what is waited for
        if (!(ok = tc::warp_wait(&sm.full[stage], parity))) break;
        if (!(ok = tc::warp_wait(&sm.sum_empty[buf], buf_parity))) break;
        tc::fence_after_sync();
        if (lane == 0) {
          for (int k = 0; k < 4; ++k)  // 32 bytes of k an instruction
            tc::mma_e4m3(tmem + buf * kWideCols, dx + 2 * k, dw + 2 * k, instruction, k > 0);
          tc::mma_commit(staging::smem_addr(&sm.empty[stage]));
          tc::mma_commit(staging::smem_addr(&sm.sum_full[buf]));
        }
        __syncwarp();
        stage += 2;
        if (stage >= uint32_t(stages)) stage -= stages, parity ^= 1;
        buf_parity ^= 1;
      }
      if (!ok && lane == 0) give_up(a.status, kStatusMatrixWait);
    }
  } else {  // sums
    tc::registers_up<kWideSumRegisters>();
    const int quarter = warp & 3, part = warp >> 2;
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16) + part * kWideWarpCols;
    unsigned char* out = sm.out[warp];
    float* scales = sm.scales[warp];
    float next_x[8], next_w = 0.0f;  // scales of the 8 blocks to come
    auto fetch = [&](const Tile& tile, int b0) {
      const int b = b0 + lane % kScaleBlocks;
      const int row0 = tile.row + quarter * 32 + lane / kScaleBlocks;
      const int block = min((tile.n0 + part * kWideWarpCols) / kBlock, a.col_blocks - 1);
      if (b >= b1) return;
      next_w = a.ws[(int64_t(tile.e) * a.col_blocks + block) * a.ldws + b];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        next_x[i] = a.xs[int64_t(min(row0 + 4 * i, a.tokens - 1)) * a.ldxs + b];
    };
    uint32_t buf = 0, parity = 0;
    bool ok = true;
    Tile tile;
    if (unit < total) {
      tile = Tile(table, a.nexperts, unit, kRows, kWideCols);
      fetch(tile, b0);
    }
    for (int t = unit; ok && t < total; t += units) {
      const Tile following(table, a.nexperts, min(t + units, total - 1), kRows, kWideCols);
      const int row0 = tile.row + quarter * 32;
      const int col0 = tile.n0 + part * kWideWarpCols;
      uint64_t acc[kWideWarpCols / 2];
#pragma unroll
      for (int i = 0; i < kWideWarpCols / 2; ++i) acc[i] = 0;
      for (int b = b0; b < b1; ++b) {
        const int step = b - b0;
        if (step % kScaleBlocks == 0) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            scales[(4 * i + lane / kScaleBlocks) * kScalePitch + lane % kScaleBlocks] =
                next_x[i] * next_w;
          __syncwarp();
          const bool last = b + kScaleBlocks >= b1;
          fetch(last ? following : tile, last ? b0 : b + kScaleBlocks);
        }
        const uint32_t s = __float_as_uint(scales[lane * kScalePitch + step % kScaleBlocks]);
        const uint64_t scale = tc::pack2(s, s);
        if (!(ok = tc::warp_wait(&sm.sum_full[buf], parity))) break;
        tc::fence_after_sync();
        const uint32_t from = lanes + buf * kWideCols;
        uint32_t v[2][16];
        tc::tmem_load16(from, v[0]);
#pragma unroll
        for (int c = 0; c < kWideWarpCols / 16; ++c) {
          tc::tmem_wait(v[c & 1]);
          if (c + 1 < kWideWarpCols / 16) tc::tmem_load16(from + 16 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            acc[8 * c + i] =
                tc::fma2(tc::pack2(v[c & 1][2 * i], v[c & 1][2 * i + 1]), scale, acc[8 * c + i]);
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) staging::mbar_arrive(&sm.sum_empty[buf]);
        if (++buf == 2) buf = 0, parity ^= 1;
      }
      if (ctas > 1) {  // one tile a cluster
        tc::cluster_sync();  // every CTA is done with its stages
        // [slot of a chunk][CTA][4 columns][row][4]: a warp's store is 512 bytes in a row
        const uint32_t at = data + rank * kSplitChunkBytes + (quarter * 32 + lane) * 16;
        const int chunk0 = part * (kWideWarpCols / kSplitChunk);
        uint32_t owner = chunk0 % ctas, to = at + chunk0 / ctas * ctas * kSplitChunkBytes;
        const bool any = row0 < tile.end;
#pragma unroll
        for (int i = 0; i < kWideWarpCols / kSplitChunk; ++i) {
          const uint32_t there = tc::in_cta(to, owner);
          if (any) {
#pragma unroll
            for (int j = 0; j < kSplitChunk / 4; ++j)
              tc::store_cluster16(there + j * (kRows * 16), acc[i * (kSplitChunk / 2) + 2 * j],
                                  acc[i * (kSplitChunk / 2) + 2 * j + 1]);
          }
          if (++owner == ctas) owner = 0, to += ctas * kSplitChunkBytes;
        }
        tc::cluster_sync();
        const float4* sums = reinterpret_cast<const float4*>(
            dynamic + wide_stages_at(ExpertTable::bytes(a.nexperts)));
        Y* y = static_cast<Y*>(a.y) + int64_t(tile.row) * a.ldy + tile.n0;
        const int rows = ok ? min(tile.end - tile.row, kRows) : 0, cols = a.n - tile.n0;
        for (int chunk = int(rank), slot = 0; chunk < kWideCols / kSplitChunk; chunk += ctas, slot += ctas) {
          const float4* chunks = sums + slot * (kSplitChunkBytes / 16);
          if (a.aligned_y && (chunk + 1) * kSplitChunk <= cols) {  // 8 columns of a row a thread
            const int r = threadIdx.x % kRows, h = threadIdx.x / kRows * 8;
            float sum[8] = {};
            const float4* from = chunks + h / 4 * kRows + r;
            for (int q = 0; q < int(ctas); ++q, from += kSplitChunkBytes / 16) {
              const float4 lo = from[0], hi = from[kRows];
              sum[0] += lo.x, sum[1] += lo.y, sum[2] += lo.z, sum[3] += lo.w;
              sum[4] += hi.x, sum[5] += hi.y, sum[6] += hi.z, sum[7] += hi.w;
            }
            __align__(16) Y v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = from_float<Y>(sum[j]);
            uint4* to = reinterpret_cast<uint4*>(y + int64_t(r) * a.ldy + chunk * kSplitChunk + h);
            if (r < rows) {
#pragma unroll
              for (int j = 0; j < int(sizeof(Y)) / 2; ++j) to[j] = reinterpret_cast<const uint4*>(v)[j];
            }
          } else {  // neighbouring lanes on neighbouring columns
            const int c = threadIdx.x % kSplitChunk, col = chunk * kSplitChunk + c;
            for (int r = threadIdx.x / kSplitChunk; r < rows; r += 32 * kWideSumWarps / kSplitChunk) {
              const float* from = reinterpret_cast<const float*>(chunks + c / 4 * kRows + r) + c % 4;
              float sum = 0.0f;
              for (int q = 0; q < int(ctas); ++q) sum += from[q * (kSplitChunkBytes / 4)];
              if (col < cols) y[int64_t(r) * a.ldy + col] = from_float<Y>(sum);
            }
          }
        }
        break;
      }
      if (!ok) break;
      if (a.aligned_y == 32 && col0 + kWideWarpCols <= a.n) {
        // whole sectors from every lane: few instructions, which are new to the SM at the end
        // of its first tile
        if (row0 + lane < tile.end) {
          Y* to = static_cast<Y*>(a.y) + int64_t(row0 + lane) * a.ldy + col0;
          constexpr int kVec = 32 / int(sizeof(Y));
#pragma unroll
          for (int j = 0; j < kWideWarpCols / kVec; ++j) tc::store32(to + j * kVec, acc + j * (kVec / 2));
        }
        tile = following;
        continue;
      }
      // through shared memory, so that neighbouring lanes store neighbouring columns
      constexpr int kChunk = kOutRow / int(sizeof(Y));  // columns of a round
      constexpr int kVec = 16 / int(sizeof(Y));
      static_assert(32 % kChunk == 0, "a lane keeps its column");
      Y* y = static_cast<Y*>(a.y);
      // (whose code is there once for all rounds)
#pragma unroll 1
      for (int round = 0; round < kWideWarpCols / kChunk; ++round) {
#pragma unroll
        for (int rr = 0; rr < kWideWarpCols / kChunk; ++rr) {
          if (rr != round) continue;
#pragma unroll
          for (int j = 0; j < kOutRow / 16; ++j) {
            __align__(16) Y vec[kVec];
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) {
              const float2 f = tc::unpack2(acc[(rr * kChunk + j * kVec) / 2 + i]);
              vec[2 * i] = from_float<Y>(f.x);
              vec[2 * i + 1] = from_float<Y>(f.y);
            }
            *reinterpret_cast<uint4*>(out + lane * kOutPitch + j * 16) =
                *reinterpret_cast<const uint4*>(vec);
          }
        }
        __syncwarp();
        const int c0 = col0 + round * kChunk;
        if (a.aligned_y) {
#pragma unroll
          for (int i = 0; i < kOutRow / 16; ++i) {
            constexpr int kLanes = kOutRow / 16;  // lanes of a row
            const int r = i * (32 / kLanes) + lane / kLanes, c = c0 + lane % kLanes * kVec;
            const uint4 v = *reinterpret_cast<const uint4*>(out + r * kOutPitch + lane % kLanes * 16);
            if (row0 + r < tile.end && c < a.n) {
              Y* to = y + int64_t(row0 + r) * a.ldy + c;
              if (c + kVec <= a.n) {
                *reinterpret_cast<uint4*>(to) = v;
              } else {
                const Y* e = reinterpret_cast<const Y*>(&v);
                for (int k = 0; k < a.n - c; ++k) to[k] = e[k];
              }
            }
          }
        } else {
          // eight loads, then eight stores: a store to y would hold up loads behind it
          for (int i0 = lane; i0 < 32 * kChunk; i0 += 8 * 32) {
            Y v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int e = i0 + 32 * i;
              v[i] = *reinterpret_cast<const Y*>(out + e / kChunk * kOutPitch + e % kChunk * sizeof(Y));
            }
            Y* to = y + int64_t(row0 + i0 / kChunk) * a.ldy + c0 + i0 % kChunk;
            const bool inside = c0 + i0 % kChunk < a.n;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (inside && row0 + (i0 + 32 * i) / kChunk < tile.end)
                to[int64_t(32 / kChunk * i) * a.ldy] = v[i];
          }
        }
        __syncwarp();
      }
      tile = following;
    }
    if (!ok && lane == 0) give_up(a.status, kStatusSumWait);
  }
  __syncwarp();
  if (ctas > 1 && unit < total && warp >= kWideSumWarps) {  // as the summing warps
    tc::cluster_sync();
    tc::cluster_sync();
  }
  tc::fence_before_sync();
  tc::cluster_sync();
  if (warp == kWideSumWarps + 1) tc::tmem_free(tmem, 512);
}

// ----------------------------------------------------------------------------- narrow
// One tile of 128 features x NT tokens a CTA: four summing warps, a loading warp and two
// matrix warps.  `split` CTAs of a cluster take a share of the blocks of k each and send
// their sums through distributed shared memory to the CTA that adds up the column, in rank
// order.  Bound by reading w where there is much of it (1024 tokens over 256 experts of
// [256, 7168]: 68 us, 7.0 TB/s), by latencies where there is little (1 x 2688 x 7168: 8.2
// us, of which 3 us are the loads; 777 x 2867 x 819 to float32 in 64-token tiles 8.3 to
// 10.3 us).  Four stages of loads and four accumulators keep both matrix warps'
// instructions in flight: a group of four for so few tokens takes 560 clocks by itself
// whatever their number.
constexpr int kMatrixWarps = 2;
constexpr int kNarrowThreads = 32 * (5 + kMatrixWarps);
constexpr int kNarrowStages = 4, kNarrowBufs = 4;
static_assert(kNarrowStages % kMatrixWarps == 0 && kNarrowBufs % kMatrixWarps == 0,
              "a stage and an accumulator belong to one matrix warp each");

template <int NT>
struct NarrowSmem {
  static constexpr int kStageBytes = kTileBytes + NT * kBlock;
  alignas(1024) unsigned char stages[kNarrowStages][kStageBytes];
  alignas(16) float scales[2][kScaleBlocks][NT + 4];  // no bank conflicts where they are written
  uint64_t full[kNarrowStages], empty[kNarrowStages], sum_full[kNarrowBufs], sum_empty[kNarrowBufs];
  uint32_t tmem;
  // behind it: the expert table and, with several CTAs a tile, the sums that this CTA adds up:
  // float4 (4 tokens) [chunk of 4 tokens][CTA][kRows]
  static constexpr int kChunks = NT / 4, kChunkBytes = 16 * kRows;
  __host__ __device__ static constexpr size_t sum_bytes(int split) {
    return size_t((kChunks + split - 1) / split * split) * kChunkBytes;
  }
  __host__ __device__ static constexpr size_t sums_at(size_t table_bytes) {
    return (sizeof(NarrowSmem) + table_bytes + 15) / 16 * 16;
  }
};
static_assert(NarrowSmem<64>::sums_at(kTableMost) + NarrowSmem<64>::sum_bytes(7) <= kSmemMost, "7 needs the most");

template <int NT, typename Y>
__global__ void __launch_bounds__(kNarrowThreads, 2)
    narrow_kernel(const __grid_constant__ CUtensorMap map_x,
                  const __grid_constant__ CUtensorMap map_w, const __grid_constant__ MatmulArgs a,
                  const int split) {
  using S = NarrowSmem<NT>;
  extern __shared__ __align__(1024) unsigned char dynamic[];
  NarrowSmem<NT>& sm = *reinterpret_cast<NarrowSmem<NT>*>(dynamic);
  ExpertTable table(reinterpret_cast<char*>(dynamic + sizeof(NarrowSmem<NT>)), a.nexperts);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float4* sums = reinterpret_cast<float4*>(dynamic + NarrowSmem<NT>::sums_at(ExpertTable::bytes(a.nexperts)));
  const int rank = int(blockIdx.x) % split, index = int(blockIdx.x) / split;

  if (split > 1) tc::cluster_arrive();  // the others run before this CTA writes to them
  if (threadIdx.x == 128) {
    tc::prefetch_map(&map_x);
    tc::prefetch_map(&map_w);
  }
  table.build(a, NT);
  __syncthreads();
  if (index >= table.tiles[a.nexperts]) {  // the whole cluster
    if (split > 1) tc::cluster_wait();
    return;
  }
  const Tile tile(table, a.nexperts, index, NT, kRows);
  const int b0 = int(int64_t(a.blocks) * rank / split);
  const int b1 = int(int64_t(a.blocks) * (rank + 1) / split);
  const int cols = min(NT, tile.end - tile.row);
  auto load = [&](int b, uint32_t stage) {
    mbar_arrive_expect(&sm.full[stage], S::kStageBytes);
    const uint32_t bar = staging::smem_addr(&sm.full[stage]);
    const uint32_t dst = staging::smem_addr(sm.stages[stage]);
    tc::load_box(dst, &map_w, bar, b * kBlock, tile.n0, tile.e);
    tc::load_box(dst + kTileBytes, &map_x, bar, b * kBlock, tile.row, 0);
  };
  if (warp == 4 && lane == 0) {  // the first loads wait for nothing else
    for (int i = 0; i < kNarrowStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < kNarrowBufs; ++i) {
      mbar_init(&sm.sum_full[i], 1);
      mbar_init(&sm.sum_empty[i], 4);
    }
    tc::fence_barrier_init();
    for (int i = 0; i < kNarrowStages && b0 + i < b1; ++i) load(b0 + i, i);
  }
  __syncwarp();
  if (warp == 5) tc::tmem_alloc(&sm.tmem, kNarrowBufs * NT);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (split > 1) tc::cluster_wait();
  const uint32_t tmem = sm.tmem;

  if (warp == 4) {  // loads
    uint32_t stage = 0, parity = 0;
    bool ok = true;
    for (int b = b0 + kNarrowStages; b < b1; ++b) {
      if (!(ok = tc::warp_wait(&sm.empty[stage], parity))) break;
      if (lane == 0) load(b, stage);
      __syncwarp();
      if (++stage == kNarrowStages) stage = 0, parity ^= 1;
    }
    // every matrix instruction has let go of its stage before this CTA may end
    for (int i = 0; ok && i < kNarrowStages && i < b1 - b0; ++i) {
      ok = tc::warp_wait(&sm.empty[stage], parity);
      if (++stage == kNarrowStages) stage = 0, parity ^= 1;
    }
    if (!ok && lane == 0) give_up(a.status, kStatusLoadWait);
  } else if (warp >= 5) {  // matrix instructions, every other block
    constexpr uint32_t instruction = tc::e4m3_instruction(kRows, NT);
    bool ok = true;
    for (int i = warp - 5; i < b1 - b0; i += kMatrixWarps) {
      const uint32_t stage = i % kNarrowStages, buf = i % kNarrowBufs;
      if (!(ok = tc::warp_wait(&sm.sum_empty[buf], (i / kNarrowBufs & 1) ^ 1))) break;
      if (!(ok = tc::warp_wait(&sm.full[stage], i / kNarrowStages & 1))) break;
      tc::fence_after_sync();
      if (lane == 0) {
        const uint32_t src = staging::smem_addr(sm.stages[stage]);
        const uint64_t dw = tc::tile_desc(src), dx = tc::tile_desc(src + kTileBytes);
        for (int k = 0; k < 4; ++k)
          tc::mma_e4m3(tmem + buf * NT, dw + 2 * k, dx + 2 * k, instruction, k > 0);
        tc::mma_commit(staging::smem_addr(&sm.sum_full[buf]));
        tc::mma_commit(staging::smem_addr(&sm.empty[stage]));
      }
      __syncwarp();
    }
    if (!ok && lane == 0) give_up(a.status, kStatusMatrixWait);
  } else {  // sums: a thread has one feature of every token
    const uint32_t lanes = tmem + (uint32_t(warp * 32) << 16);
    const float* ws = a.ws + (int64_t(tile.e) * a.col_blocks + tile.n0 / kBlock) * a.ldws;
    // The four warps fetch the scales of every token for 8 blocks at a time, a sector a
    // token, and share the products of both scales in shared memory.
    float next_x[NT / 16], next_w = 0.0f;
    auto fetch = [&](int begin) {
      const int b = begin + lane % kScaleBlocks;
      if (b >= b1) return;
      next_w = ws[b];
#pragma unroll
      for (int i = 0; i < NT / 16; ++i)
        next_x[i] =
            a.xs[int64_t(min(tile.row + 16 * i + int(threadIdx.x) / kScaleBlocks, a.tokens - 1)) * a.ldxs + b];
    };
    fetch(b0);
    uint64_t acc[NT / 2];
#pragma unroll
    for (int i = 0; i < NT / 2; ++i) acc[i] = 0;
    uint32_t buf = 0, parity = 0;
    bool ok = true;
    for (int b = b0; b < b1; ++b) {
      const int step = b - b0;
      if (step % kScaleBlocks == 0) {
        float(*to)[NT + 4] = sm.scales[step / kScaleBlocks & 1];
#pragma unroll
        for (int i = 0; i < NT / 16; ++i)
          to[lane % kScaleBlocks][16 * i + threadIdx.x / kScaleBlocks] = next_x[i] * next_w;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        fetch(b + kScaleBlocks);
      }
      const float* scales = sm.scales[step / kScaleBlocks & 1][step % kScaleBlocks];
      // no way out of the loop before its end: the other warps wait at the barrier above
      ok = ok && tc::warp_wait(&sm.sum_full[buf], parity);
      tc::fence_after_sync();
      const uint32_t from = lanes + buf * NT;
      uint32_t v[2][16];
      tc::tmem_load16(from, v[0]);
#pragma unroll
      for (int c = 0; c < NT / 16; ++c) {
        tc::tmem_wait(v[c & 1]);
        if (c + 1 < NT / 16) tc::tmem_load16(from + 16 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const ulonglong2 s = reinterpret_cast<const ulonglong2*>(scales)[c * 4 + i];
          acc[c * 8 + 2 * i] = tc::fma2(tc::pack2(v[c & 1][4 * i], v[c & 1][4 * i + 1]), s.x,
                                        acc[c * 8 + 2 * i]);
          acc[c * 8 + 2 * i + 1] = tc::fma2(tc::pack2(v[c & 1][4 * i + 2], v[c & 1][4 * i + 3]), s.y,
                                            acc[c * 8 + 2 * i + 1]);
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) staging::mbar_arrive(&sm.sum_empty[buf]);
      if (++buf == kNarrowBufs) buf = 0, parity ^= 1;
    }
    if (!ok && lane == 0) give_up(a.status, kStatusSumWait);
    const int feature = warp * 32 + lane;
    Y* y = static_cast<Y*>(a.y) + int64_t(tile.row) * a.ldy + tile.n0 + feature;
    if (split == 1) {
      if (ok && tile.n0 + feature < a.n) {
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) {
          const float2 f = tc::unpack2(acc[i]);
          if (2 * i < cols) y[2 * i * a.ldy] = from_float<Y>(f.x);
          if (2 * i + 1 < cols) y[(2 * i + 1) * a.ldy] = from_float<Y>(f.y);
        }
      }
    } else {
      // chunk i to CTA i % split; 512 bytes a warp's store (a token at a time, 128 bytes: 32
      // tokens x [2688, 4096] 8.3 us, so 6.2 us)
      const uint32_t at = staging::smem_addr(sums + rank * kRows + feature);
#pragma unroll
      for (int i = 0; i < S::kChunks; ++i)
        if (4 * i < cols)
          tc::store_cluster16(tc::in_cta(at + i / split * split * S::kChunkBytes, i % split), acc[2 * i],
                              acc[2 * i + 1]);
    }
  }
  __syncwarp();
  if (split > 1) {
    tc::cluster_sync();
    if (warp < 4 && tile.n0 + int(threadIdx.x) < a.n) {
      Y* y = static_cast<Y*>(a.y) + int64_t(tile.row) * a.ldy + tile.n0 + threadIdx.x;
      for (int i = rank; 4 * i < cols; i += split) {
        const float4* from = sums + i / split * split * kRows + threadIdx.x;
        float4 sum = {};
#pragma unroll
        for (int r = 0; r < kMostSplit; ++r) {
          if (r >= split) continue;
          const float4 v = from[r * kRows];
          sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
        Y* to = y + int64_t(4 * i) * a.ldy;
        to[0] = from_float<Y>(sum.x);
        if (4 * i + 1 < cols) to[a.ldy] = from_float<Y>(sum.y);
        if (4 * i + 2 < cols) to[2 * a.ldy] = from_float<Y>(sum.z);
        if (4 * i + 3 < cols) to[3 * a.ldy] = from_float<Y>(sum.w);
      }
    }
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 5) tc::tmem_free(tmem, kNarrowBufs * NT);
}

// An inner size of zero: the rows of experts get zeros.
template <typename Y>
__global__ void zero_kernel(const MatmulArgs a) {
  __shared__ int most;
  if (threadIdx.x == 0) most = 0;
  __syncthreads();
  int first = 0, end = a.tokens;
  if (a.offsets != nullptr) {
    first = min(max(a.offsets[0], 0), a.tokens);
    for (int e = threadIdx.x; e <= a.nexperts; e += blockDim.x)  // one below an earlier one counts as that
      atomicMax(&most, min(a.offsets[e], a.tokens));
    __syncthreads();
    end = most;
  }
  for (int r = first + int(blockIdx.x); r < end; r += int(gridDim.x))
    for (int c = threadIdx.x; c < a.n; c += blockDim.x)
      static_cast<Y*>(a.y)[int64_t(r) * a.ldy + c] = from_float<Y>(0.0f);
}

// ------------------------------------------------------------------------------- host
// [planes][rows][pitch] bytes, of which k a row count; boxes of 128 bytes x box_rows rows,
// zeros beyond every edge.
reshard_status_t tile_map(CUtensorMap* map, const void* base, int64_t k, int64_t rows, int64_t planes,
                          int64_t pitch, int box_rows) {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> entry{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 encode = entry.load(std::memory_order_acquire);
  if (!encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    const cudaError_t ce =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (ce != cudaSuccess || found != cudaDriverEntryPointSuccess || !fn)
      return fail(RESHARD_ERR_CUDA, std::string("cuTensorMapEncodeTiled: ") + cudaGetErrorString(ce));
    encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    entry.store(encode, std::memory_order_release);
  }
  const cuuint64_t dims[3] = {cuuint64_t(k), cuuint64_t(rows), cuuint64_t(planes)};
  const cuuint64_t strides[2] = {cuuint64_t(pitch), cuuint64_t(pitch) * cuuint64_t(rows)};
  const cuuint32_t box[3] = {kBlock, cuuint32_t(box_rows), 1}, steps[3] = {1, 1, 1};
  auto encoded = [&] {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box,
                  steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encoded();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {
    // a host thread's first call: the driver, unlike the runtime, does not make its device's
    // context current
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = encoded();
  }
  if (r != CUDA_SUCCESS)
    return fail(RESHARD_ERR_CUDA, "cuTensorMapEncodeTiled: error " + std::to_string(int(r)));
  return RESHARD_OK;
}

// How many clusters of `split` CTAs are on the device at a time: fewer than its SMs divided
// by the split, since a cluster lies in one part of the GPU (8 CTAs of an SM each: 15, not
// 19).  Asked for once a device and kernel: the record is the kernel's own (kernels differ in
// what fits, though not in their type), so that no call changes what another one chooses.
template <auto Kernel>
int resident_clusters(int dev, unsigned threads, size_t smem, int split) {
  constexpr int kDevices = 16;
  static std::atomic<int> known[kDevices][kMostSplit + 1];
  if (dev < kDevices) {
    const int n = known[dev][split].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(split));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {unsigned(split), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (allow_smem<Kernel, kSmemMost>(dev) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();  // an estimate is not worth an error: the launch reports its own
    return 1;
  }
  if (dev < kDevices) known[dev][split].store(n, std::memory_order_relaxed);
  return n > 0 ? n : 1;
}

// Which kernel a call takes: `tokens` of a tile (narrow with 16, 32 or 64, wide with 128),
// `split` CTAs a tile, and `units` of them: tiles, or for wide undivided the CTAs that go
// through the tiles.
struct Path {
  int tokens, split;
  int64_t units;
};

// ns that the sums of a tile's tokens take through a cluster.
inline int64_t sums_way(int64_t tokens) { return 750 + 18 * tokens; }

// Experts that can have rows, where rows are sorted by expert.
inline int64_t experts_with_rows(const MatmulArgs& a) {
  return !a.offsets ? 0 : a.nexperts < a.tokens ? a.nexperts : a.tokens;
}
// The most tiles of rows x cols that there can be.
inline int64_t most_tiles(const MatmulArgs& a, int64_t rows, int64_t cols) {
  return cdiv(a.n, cols) * (a.offsets ? a.tokens / rows + experts_with_rows(a) : cdiv(a.tokens, rows));
}

template <int NT, typename Y>
Path narrow_path(const MatmulArgs& a, int64_t each, int dev, int64_t sms) {
  const int64_t tiles = most_tiles(a, NT, kRows);
  // CTAs a tile, within one wave (a second one would cost more than longer shares) and with two
  // blocks each: the least of a share's blocks and, with several CTAs, the sums' way to the CTA
  // that adds them up, in ns.  (32 tokens' k = 512 takes 4.5 us undivided, longer by two CTAs;
  // k = 4096 10.7 us and, by eight, 6.2 us; one token's k = 1024 5.0 us and, by four, 4.2 us.)
  const int64_t block = NT == 64 ? 450 : 210, way = sums_way(each < NT ? each : NT);
  int64_t best = a.blocks * block;
  int split = 1;
  for (int s = 2; s <= kMostSplit; ++s) {
    const int64_t cost = cdiv(a.blocks, s) * block + way;
    if (cost < best && a.blocks >= 2 * s && tiles * s <= 2 * sms &&
        tiles <= resident_clusters<narrow_kernel<NT, Y>>(
                     dev, kNarrowThreads, NarrowSmem<NT>::sums_at(0) + NarrowSmem<NT>::sum_bytes(s), s))
      best = cost, split = s;
  }
  return {NT, split, tiles};
}

// Four stages of the wide kernel, which a split needs for its sums.
inline bool wide_room(const MatmulArgs& a) {
  return wide_stages_at(ExpertTable::bytes(a.nexperts)) + kWideStages * kWideStageBytes <= kSmemMost;
}

template <typename Y>
Path matmul_path(const MatmulArgs& a, int dev, int64_t sms) {
  // Few tokens (of an expert, on average; experts differ): reading w is all that counts.
  const int64_t each = cdiv(a.tokens, a.nexperts);
  if (each <= (a.offsets ? 4 : 16)) return narrow_path<16, Y>(a, each, dev, sms);
  if (each <= (a.offsets ? 8 : 32)) return narrow_path<32, Y>(a, each, dev, sms);

  // Otherwise the least of these estimates in ns, fitted to 20 sizes from 64 x 7168 x 7168 to
  // 4096 x 4096 x 4096 within 15%: a kernel's start and end, and a time for each block of k
  // that the CTAs of an SM go through one after the other (w from HBM costs all the same).
  // Tiles of `rows` tokens: an expert's last one may be short, half of one on average.
  auto tiles = [&](int64_t rows, int64_t cols) {
    return cdiv(a.n, cols) * cdiv(2 * cdiv(a.tokens, rows) + experts_with_rows(a), 2);
  };
  const int64_t blocks = a.blocks, stray = a.aligned_y == 32 ? 0 : 6000;  // rows off the sectors
  const int64_t small = tiles(64, kRows), large = tiles(kRows, kWideCols);
  int64_t best = 5500 + cdiv(small, 2 * sms) * blocks * (small > sms ? 650 : 450);
  for (int s = 2; s <= kMostSplit; ++s) {
    const int64_t cost = 5500 + cdiv(blocks, s) * 450 + sums_way(64);
    if (cost < best && blocks >= 2 * s && small * s <= sms) best = cost;
  }
  int split = 0;  // 0: narrow, else CTAs a tile of 128 tokens
  const bool room = wide_room(a);
  for (int s = 1; s <= kMostSplit; ++s) {
    if (s > 1 && (!room || blocks < 2 * s || large * s > sms ||
                  large > resident_clusters<wide_kernel<Y>>(dev, kWideThreads, kSmemMost, s)))
      continue;
    const int64_t cost = s == 1 ? 7500 + cdiv(large, sms) * (blocks * 540 + 1500 + stray)
                                : 10500 + cdiv(blocks, s) * 500;
    if (cost < best) best = cost, split = s;
  }
  if (split == 0) return narrow_path<64, Y>(a, each, dev, sms);
  const int64_t units = most_tiles(a, kRows, kWideCols);
  return {kRows, split, split == 1 && units > sms ? sms : units};
}

struct Operands {
  const void *x, *w;
  int64_t ldx, ldw, k;
};

reshard_status_t tile_maps(CUtensorMap* map_x, CUtensorMap* map_w, const MatmulArgs& a, const Operands& o,
                           int rows) {
  const reshard_status_t st = tile_map(map_x, o.x, o.k, a.tokens, 1, o.ldx, rows);
  return st == RESHARD_OK ? tile_map(map_w, o.w, o.k, a.n, a.nexperts, o.ldw, kRows) : st;
}

template <typename Y>
reshard_status_t launch_wide(MatmulArgs& a, const Operands& o, const Path& p, int dev, cudaStream_t stream) {
  CUtensorMap map_x, map_w;
  const reshard_status_t st = tile_maps(&map_x, &map_w, a, o, kRows);
  if (st != RESHARD_OK) return st;
  a.ntiles = int32_t(cdiv(a.n, kWideCols));
  int stages = wide_room(a) ? kWideStages : 2;
  const size_t smem = wide_stages_at(ExpertTable::bytes(a.nexperts)) + size_t(stages) * kWideStageBytes;
  void* args[] = {&map_x, &map_w, &a, &stages};
  return launch<wide_kernel<Y>, kSmemMost>("reshard_fp8_matmul", dev,
                                           {p.units * p.split, kWideThreads, smem, p.split, stream}, args);
}
static_assert(split_chunks(7) * kSplitChunkBytes <= kWideStages * kWideStageBytes, "7 needs the most");

template <int NT, typename Y>
reshard_status_t launch_narrow(MatmulArgs& a, const Operands& o, const Path& p, int dev, cudaStream_t stream) {
  if (p.units * p.split >= int64_t(1) << 31)
    return fail(RESHARD_ERR_UNSUPPORTED, "reshard_fp8_matmul: too many tiles");
  CUtensorMap map_x, map_w;
  const reshard_status_t st = tile_maps(&map_x, &map_w, a, o, NT);
  if (st != RESHARD_OK) return st;
  a.ntiles = int32_t(cdiv(a.n, kRows));
  const size_t table = ExpertTable::bytes(a.nexperts);
  const size_t smem = p.split > 1 ? NarrowSmem<NT>::sums_at(table) + NarrowSmem<NT>::sum_bytes(p.split)
                                  : sizeof(NarrowSmem<NT>) + table;
  int split = p.split;
  void* args[] = {&map_x, &map_w, &a, &split};
  return launch<narrow_kernel<NT, Y>, kSmemMost>("reshard_fp8_matmul", dev,
                                                 {p.units * split, kNarrowThreads, smem, split, stream}, args);
}

// The current device's path for these sizes.
template <typename Y>
reshard_status_t path_here(const MatmulArgs& a, int* dev, Path* p) {
  int sms = 0;
  cudaError_t ce = cudaGetDevice(dev);
  if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, *dev);
  if (ce != cudaSuccess)
    return fail(RESHARD_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(ce));
  *p = matmul_path<Y>(a, *dev, sms);
  return RESHARD_OK;
}

template <typename Y>
reshard_status_t launch_matmul(MatmulArgs& a, const Operands& o, cudaStream_t stream) {
  if (a.blocks == 0) {
    zero_kernel<Y><<<unsigned(a.tokens < 1024 ? a.tokens : 1024), 256, 0, stream>>>(a);
    return launched("reshard_fp8_matmul");
  }
  int dev = 0;
  Path p;
  reshard_status_t st = path_here<Y>(a, &dev, &p);
  if (st == RESHARD_OK) st = device_status_word(&a.status);
  if (st != RESHARD_OK) return st;
  if (p.tokens == 16) return launch_narrow<16, Y>(a, o, p, dev, stream);
  if (p.tokens == 32) return launch_narrow<32, Y>(a, o, p, dev, stream);
  if (p.tokens == 64) return launch_narrow<64, Y>(a, o, p, dev, stream);
  return launch_wide<Y>(a, o, p, dev, stream);
}

// The checks of sizes, offsets and y, and what of the arguments follows from them.
reshard_status_t matmul_args(const int32_t* offsets, int64_t nexperts, int64_t tokens, int64_t n, int64_t k,
                             void* y, int32_t ydtype, int64_t ldy, MatmulArgs* a) {
  if (!float_dtype(ydtype)) return fail(RESHARD_ERR_INVALID_ARG, "ydtype must be BF16, FP16 or FP32");
  if (tokens < 0 || n < 0 || k < 0 || nexperts < 1)
    return fail(RESHARD_ERR_INVALID_ARG, "negative size");
  if (!offsets && nexperts != 1)
    return fail(RESHARD_ERR_INVALID_ARG, "several experts need offsets");
  if (nexperts > RESHARD_MAX_EXPERTS) return fail(RESHARD_ERR_UNSUPPORTED, "too many experts");
  constexpr int64_t kMost = (int64_t(1) << 31) - 1024;  // rounding up to tiles stays in 32 bits
  if (tokens >= kMost || n >= kMost || k >= kMost || nexperts * n >= kMost)
    return fail(RESHARD_ERR_UNSUPPORTED, "size of nearly 2^31 or more");
  if (tokens == 0 || n == 0) return RESHARD_OK;
  if (ldy < n) return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  if (!y) return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  if (!aligned(offsets, 4) || !aligned(y, dtype_size(ydtype)))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
  *a = {};
  a->offsets = offsets;
  a->nexperts = int32_t(nexperts);
  a->tokens = int32_t(tokens);
  a->n = int32_t(n);
  a->blocks = int32_t(cdiv(k, 128));
  a->col_blocks = int32_t(cdiv(n, 128));
  a->y = y;
  a->ldy = ldy;
  const int64_t pitch = ldy * dtype_size(ydtype);
  a->aligned_y = aligned(y, 32) && pitch % 32 == 0 ? 32 : aligned(y, 16) && pitch % 16 == 0 ? 16 : 0;
  return RESHARD_OK;
}

}  // namespace
}  // namespace rs

using rs::fail;

extern "C" reshard_status_t reshard_fp8_matmul(const void* x, int64_t ldx, const float* xs,
                                               int64_t ldxs, const void* w, int64_t ldw,
                                               const float* ws, int64_t ldws,
                                               const int32_t* offsets, int64_t nexperts,
                                               int64_t tokens, int64_t n, int64_t k, void* y,
                                               int32_t ydtype, int64_t ldy, void* stream) {
  rs::TraceRange trace("op.fp8_matmul");
  rs::MatmulArgs a;
  const reshard_status_t st = rs::matmul_args(offsets, nexperts, tokens, n, k, y, ydtype, ldy, &a);
  if (st != RESHARD_OK || tokens == 0 || n == 0) return st;
  if (ldx < k || ldw < k || ldxs < a.blocks || ldws < a.blocks)
    return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  if (k > 0 && (!x || !xs || !w || !ws)) return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  if (!rs::op::aligned(x, 16) || !rs::op::aligned(w, 16) || ldx % 16 != 0 || ldw % 16 != 0)
    return fail(RESHARD_ERR_INVALID_ARG, "x, w and their row pitches must be multiples of 16 bytes");
  if (!rs::op::aligned(xs, 4) || !rs::op::aligned(ws, 4))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
  a.xs = xs;
  a.ws = ws;
  a.ldxs = ldxs;
  a.ldws = ldws;
  const rs::Operands o = {x, w, ldx, ldw, k};
  return rs::op::by_dtype(ydtype, [&](auto t) {
    return rs::launch_matmul<decltype(t)>(a, o, static_cast<cudaStream_t>(stream));
  });
}

extern "C" reshard_status_t reshard_fp8_matmul_path(const int32_t* offsets, int64_t nexperts, int64_t tokens,
                                                    int64_t n, int64_t k, const void* y, int32_t ydtype,
                                                    int64_t ldy, int32_t* tile_tokens, int32_t* split) {
  if (!tile_tokens || !split) return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  rs::MatmulArgs a;
  rs::Path p = {0, 0, 0};
  reshard_status_t st =
      rs::matmul_args(offsets, nexperts, tokens, n, k, const_cast<void*>(y), ydtype, ldy, &a);
  int dev = 0;
  if (st == RESHARD_OK && tokens > 0 && n > 0 && k > 0)
    st = rs::op::by_dtype(ydtype, [&](auto t) { return rs::path_here<decltype(t)>(a, &dev, &p); });
  if (st != RESHARD_OK) return st;
  *tile_tokens = p.tokens;
  *split = p.split;
  return RESHARD_OK;
}
