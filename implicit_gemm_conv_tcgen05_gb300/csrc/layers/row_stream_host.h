// Host side of the rows streamed through shared memory: the ring's plan and its launch.
#pragma once

#include <mutex>

#include "layers_host.h"
#include "row_stream.cuh"

namespace igc {

constexpr int kStreamStatic = 2560;  // bytes for the kernels' static shared memory

// The ring for rows of which a block has at most N columns (whole units), of inputs whose elements
// have sizes[i] bytes (0: absent), with `groups` rings to a block: false where rows are too long
// for one (at least two slots).
inline bool plan_stream(const DeviceInfo& dev, int64_t N, const int (&sizes)[kStreamMats],
                        int groups, RowStream* s) {
  uint32_t at = 0;
  for (int i = 0; i < kStreamMats; ++i) {
    s->at[i] = at;
    s->size[i] = static_cast<uint32_t>(sizes[i]);
    at += static_cast<uint32_t>(N / 8 * 8 * sizes[i]);
  }
  s->slot_bytes = at > 0 ? (at + 127) / 128 * 128 : 128;  // (no whole unit: nothing to copy)
  s->plane = static_cast<uint32_t>((N / 8 * 16 + 127) / 128 * 128);
  const size_t room = dev.smem_optin - kStreamStatic;
  if (2 * s->plane >= room) return false;
  const size_t slots = (room - 2 * s->plane) / (static_cast<size_t>(groups) * s->slot_bytes);
  if (slots < 2) return false;
  s->slots = static_cast<int>(slots < kMaxSlots ? slots : kMaxSlots);
  s->wait_limit = wait_limit_ns();
  s->status = status_word();
  return true;
}

// Blocks in clusters of `cluster` (1: none), which may start while the kernel before them ends.
template <typename... Params, typename... Args>
int launch_clusters(void (*kernel)(Params...), int blocks, int cluster, int threads, size_t smem,
                    cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...) != cudaSuccess) {
    (void)cudaGetLastError();
    return IGC_ERR_CUDA;
  }
  return IGC_OK;
}

// least: bytes of dynamic shared memory that the kernel uses whatever the ring takes.
template <typename P>
int launch_stream(void (*kernel)(P, RowStream), int blocks, int cluster, int threads, int groups,
                  size_t least, cudaStream_t stream, const P& p, const RowStream& s) {
  const size_t bytes = static_cast<size_t>(2) * s.plane +
                       static_cast<size_t>(groups) * s.slots * s.slot_bytes;
  return launch_clusters(kernel, blocks, cluster, threads, bytes < least ? least : bytes, stream, p,
                         s);
}

// What a launch of a streaming kernel needs to know of it on a device, found out once.
struct StreamSetup {
  std::once_flag once[64];
  int rc[64];
  int clusters[64];  // clusters of streaming blocks (one to an SM) that the device runs at once
};

template <typename P>
int stream_setup(StreamSetup& s, void (*kernel)(P, RowStream), const DeviceInfo& dev, int cluster,
                 int threads) {
  const int d = dev.device;
  std::call_once(s.once[d], [&] {
    const int smem = static_cast<int>(dev.smem_optin) - kStreamStatic;
    s.rc[d] = IGC_ERR_CUDA;
    s.clusters[d] = dev.sm_count;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess) {
      (void)cudaGetLastError();
      return;
    }
    if (cluster > 1) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(dev.sm_count / cluster * cluster));
      cfg.blockDim = dim3(static_cast<unsigned>(threads));
      cfg.dynamicSmemBytes = static_cast<size_t>(smem);
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&s.clusters[d], kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return;
      }
    }
    s.rc[d] = s.clusters[d] > 0 ? IGC_OK : IGC_ERR_UNSUPPORTED;
  });
  return s.rc[d];
}

}  // namespace igc
