// Rows streamed through shared memory.  One block to an SM; the threads that share a row (a
// group of kLanes) walk down the rows group, group + groups, ... and keep a ring of slots, each
// filled with one row of every input by bulk copies ahead of its use, so that loads stay in
// flight while earlier rows are summed and written.  The columns' weights are kept in shared
// memory as fp32.
//
// A copy needs 16-byte boundaries and sizes: it takes the whole units of eight columns of a row.
// The columns past them (N mod 8) are one element each for the group's first threads, loaded a
// row ahead.
#pragma once

#include "layers.cuh"

namespace igc {

// Threads of a block, one to an SM: whole groups of kLanes, at most kMost.
constexpr int stream_threads(int lanes, int most) { return most / lanes * lanes; }
constexpr int kMaxSlots = 4;
constexpr int kStreamMats = 3;  // inputs of a row, at most

// The ring of one launch, in bytes: a slot is one row of each input, 16-byte aligned.
struct RowStream {
  int slots = 0;
  uint32_t slot_bytes = 0;
  uint32_t at[kStreamMats] = {};     // where an input's row starts in its slot
  uint32_t size[kStreamMats] = {};   // bytes of its elements (0: the input is absent)
  uint32_t plane = 0;                // bytes of each half of the kept weights, ahead of the ring
  uint64_t wait_limit = 0;
  unsigned long long* status = nullptr;
};

// What is on its way to a block after a wait gave up is waited for as long as this, whatever the
// limit of the waits is: a copy or a store takes microseconds.
constexpr uint64_t kLandNs = 1000000000;

// Sites of waits that gave up (device status word).
enum : uint32_t { kSiteNormBwdRow = 0x4c01, kSiteNormBwdMeet = 0x4c02, kSiteRowDrain = 0x4c03,
                kSiteMetDrain = 0x4c04 };

__device__ __forceinline__ void bulk_load(uint32_t dst_smem, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1], %2, [%3];" ::"r"(dst_smem),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// One thread: `cols` columns (whole units) of a row's inputs into a slot; from[i] is where those
// of input i start.
__device__ __forceinline__ void fill_slot(const RowStream& s, char* slot, uint64_t* bar,
                                          const char* const (&from)[kStreamMats], uint32_t cols) {
  uint32_t total = 0;
#pragma unroll
  for (int i = 0; i < kStreamMats; ++i) total += s.size[i] * cols;
  mbar_arrive_expect_tx(bar, total);
  const uint32_t to = smem_u32(slot);
  if (cols == 0) return;
#pragma unroll
  for (int i = 0; i < kStreamMats; ++i)
    if (s.size[i] != 0) bulk_load(to + s.at[i], from[i], s.size[i] * cols, bar);
}

// Eight bytes into the shared memory of a block of the cluster, counted by a barrier there
// (addresses in the cluster's shared window).
__device__ __forceinline__ void store_async_u64(uint32_t to, uint64_t v, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(to),
      "l"(v), "r"(bar)
      : "memory");
}

// Counts bytes on a barrier of this block that will not come.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(
                   smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void st_shared_cluster_u32(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// The sums that the blocks of a cluster exchange for each of a group's rows, 8 bytes from each block
// to each: two places for alternate rows, and the barriers that count the bytes.  A block sends a
// row's sums and expects the others' when it has met the row before, so no block is more than one
// row ahead of another.
template <int kCluster>
struct Meeting {
  uint64_t sums[2][kCluster];  // by block
  uint64_t bar[2];
  int sent[kCluster];  // rows that a block has sent, told by one that stopped (else all)
};

// A group's leader that stopped, once all blocks are at the end and have told the rows they sent:
// waits for the bytes on their way here.  (The closing barrier of a cluster waits for no st.async,
// and none may arrive in a block that has gone.  Ordinary stores it would wait for, but they queue
// behind the rows' own stores: 4096 x 16384 bf16 took 140 to 160 us with them, 131 with these.)
template <int kCluster>
__device__ __noinline__ void drain_meeting(Meeting<kCluster>& m, int rank,
                                              unsigned long long* status) {
  int least = m.sent[0], senders = 0;
  for (int r = 1; r < kCluster; ++r) least = min(least, m.sent[r]);
  // rows that all have sent, and so expect
  for (int k = max(least - 2, 0); k < least; ++k) {
    int none = 0;
    (void)mbar_wait(&m.bar[k & 1], static_cast<uint32_t>(k / 2) & 1u, kLandNs, &none, status,
                    kSiteMetDrain);
  }
  // the row after, that some have sent: its phase ends with what they sent
  for (int r = 0; r < kCluster; ++r) senders += m.sent[r] > least ? 1 : 0;
  if (senders == 0) return;
  uint64_t* bar = &m.bar[least & 1];
  if (m.sent[rank] > least)
    mbar_complete_tx(bar, static_cast<uint32_t>(8 * (kCluster - senders)));
  else
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(8 * senders));
  int none = 0;
  (void)mbar_wait(bar, static_cast<uint32_t>(least / 2) & 1u, kLandNs, &none, status,
                  kSiteMetDrain);
}

// The whole block: the weights of its columns (whole units; fp32, or of type kT; 1 for none) into
// shared memory, the first four of each unit in one plane and the last four in another: a warp's
// 16-byte loads then meet no bank twice.
template <int kT>
__device__ __forceinline__ void keep_weights(char* to, uint32_t plane, const void* p, int col0,
                                             int cols, bool f32) {
#pragma unroll 4
  for (int n = static_cast<int>(threadIdx.x) * 8; n < cols; n += static_cast<int>(blockDim.x) * 8) {
    float v[8];
    load_vec8<kT>(p, col0 + n, col0 + cols, f32, 1.0f, v);
    reinterpret_cast<float4*>(to)[n / 8] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(to + plane)[n / 8] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ void kept_weights(const char* from, uint32_t plane, int n,
                                             float (&w)[8]) {
  const float4 a = reinterpret_cast<const float4*>(from)[n / 8];
  const float4 b = reinterpret_cast<const float4*>(from + plane)[n / 8];
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

// After a wait gave up, the group's leader: the copies of its rows next, next + 1, ... filled - 1,
// all that may be in flight, are waited for, each for kLandNs, so that none lands after the block
// has gone or the ring has another use.  False: one never landed.
__device__ __forceinline__ bool drain_slots(const RowStream& s, uint64_t* bars, int next, int filled) {
  bool landed = true;
  for (int k = next; k < filled; ++k) {
    int none = 0;
    landed = mbar_wait(bars + k % s.slots, static_cast<uint32_t>(k / s.slots) & 1u, kLandNs, &none,
                       s.status, kSiteRowDrain) && landed;
  }
  return landed;
}

// A group's walk: rows first, first + step, ... (count of them), its slots and barriers.
struct RowWalk {
  long long first, step;
  int count;
  int t, group;
  char* slots;
  uint64_t* bars;
};

// The start of a streaming kernel: barriers and walk (ring: the dynamic shared memory).
// (kCluster blocks that share rows walk down the same ones.)
template <int kLanes, int kGroups, int kCluster>
__device__ __forceinline__ RowWalk row_walk(const RowStream& st, char* ring,
                                            uint64_t (&full)[kGroups][kMaxSlots],
                                            int* abort_flag, int* lost, int M) {
  RowWalk w;
  w.t = threadIdx.x % kLanes;
  w.group = threadIdx.x / kLanes;
  w.slots = ring + 2 * st.plane + w.group * (st.slots * st.slot_bytes);
  w.bars = full[w.group];
  if (w.t == 0) {
    for (int i = 0; i < st.slots; ++i) mbar_init(w.bars + i, 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) *abort_flag = *lost = 0;
  w.first = static_cast<long long>(blockIdx.x / kCluster) * kGroups + w.group;
  w.step = static_cast<long long>(gridDim.x / kCluster) * kGroups;
  w.count = w.first < M ? static_cast<int>((M - w.first + w.step - 1) / w.step) : 0;
  return w;
}

}  // namespace igc
