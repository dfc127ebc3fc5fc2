// Host-visible parts of chunk attention: launch shapes and the step plan.
#pragma once
#include "attn_rows.h"

namespace kvq {
namespace chunk {

constexpr int kMaxUnits = 16;   // packed K or V blocks in flight per CTA, at most
constexpr int kAuxBytes = 1024;

struct Params {
  RowAttnParams r;
  float* part_o;    // [2 * grid][rows of a CTA][D]: partial outputs, normalised
  float* part_lse;  // [2 * grid][rows of a CTA], log2 units
  int units, unit_bytes, table_bytes;  // ring of packed blocks; parameter table (per warpgroup, two of them)
  int gshift;                          // log2 of the group size
};

// Row tiles of a CTA (128 rows each), ring slots (128 x min(D, 128) fp16
// operand tiles) and shared memory of an instance.
__host__ __device__ constexpr int slot_bytes(int D) { return 128 * (D < 128 ? D : 128) * 2; }
__host__ __device__ constexpr int q_bytes(int D, int nt) { return nt * 128 * D * 2; }
__host__ __device__ constexpr int slots_of(int D, int nt) { return D > 128 ? 3 : 4; }
// Warps.  The first nt warpgroups are the softmax's, a warp on each quarter of
// the SM.  Of the others, every fourth warp (the last quarter's) has a role of
// its own -- copies, products, segments -- and the rest dequantise, four warps
// to a team: 12 of them, 8 with head dim 256, whose operand slots are few.  So
// the warp that issues the products shares its quarter, and with it the
// instruction buffer, with softmax warps only.
__host__ __device__ constexpr int teams_of(int D) { return D > 128 ? 2 : 3; }
__host__ __device__ constexpr int other_groups(int D) { return D > 128 ? 3 : 4; }
__host__ __device__ constexpr int threads_of(int D, int nt) { return 128 * (nt + other_groups(D)); }
__host__ __device__ constexpr int fixed_bytes(int D, int nt) { return q_bytes(D, nt) + slots_of(D, nt) * slot_bytes(D) + kAuxBytes; }

cudaError_t launch_i2(int head_dim, int nt, const Params& p, int grid, size_t smem, cudaStream_t stream);
cudaError_t launch_i4(int head_dim, int nt, const Params& p, int grid, size_t smem, cudaStream_t stream);

}  // namespace chunk

// Workspace of chunk attention on `grid` CTAs, and the launch.
struct ChunkPlan {
  int nt, grid;
  size_t part_lse, total;  // workspace: partial outputs first
};
ChunkPlan chunk_plan(int head_dim, int group, int bits, int batch, int total, int num_q_heads, int num_kv_heads);
cudaError_t launch_chunk_attn(const RowAttnParams& p, const ChunkPlan& plan, void* workspace, cudaStream_t stream);

}  // namespace kvq
