// What the joins of the chunk kernels are guarded by, for tests/test_chunk_join.py: the check
// of a join on the host, and one kernel whose pieces nobody takes, so that the bounded wait of
// the thread that hands them out gives up.
#include "chunk_plan.cuh"

namespace {

__global__ void __launch_bounds__(64) nobody_takes(asp::ChunkDims c, asp::ChunkJoin* joins,
                                                   uint32_t* err) {
  __shared__ asp::ChunkTasks tasks;
  __shared__ asp::ChunkStart start;
  __shared__ long long scratch[2];
  if (threadIdx.x == 0) {
    asp::chunk_tasks_init(tasks, 1);
    asp::mbar_fence_init();
  }
  __syncthreads();
  asp::chunk_plan<asp::RowCut>(c, &start, scratch, err);
  if (threadIdx.x == 0 &&
      !asp::chunk_hand_out<asp::RowCut>(tasks, c, start, joins + blockIdx.x,
                                        [](const asp::ChunkWalk<asp::RowCut>&, asp::ChunkTask&) {}))
    asp::report(err, ASP_DEVERR_TIMEOUT);
  __syncthreads();
}

}  // namespace

extern "C" int join_valid(int b, int h, int item, int pieces, int batch, int kv_heads, int cta,
                          int ctas) {
  return asp::chunk_join_valid(asp::ChunkJoin{b, h, item, pieces}, batch, kv_heads, cta, ctas);
}

// joins: [ctas][4] ints on the device; q_offsets, seq_lens: batch + 1 and batch ints; one KV head.
extern "C" int hand_out_to_nobody(const int32_t* q_offsets, const int32_t* seq_lens, int batch,
                                  int max_pages, int num_tokens, int ctas, void* joins,
                                  uint32_t* err) {
  const asp::ChunkDims c{q_offsets, seq_lens,   batch, 1, 1, 0, max_pages, 16,
                         num_tokens, asp::chunk_inverse(ctas)};
  nobody_takes<<<ctas, 64>>>(c, static_cast<asp::ChunkJoin*>(joins), err);
  return (int)cudaDeviceSynchronize();
}
