// decode_launch.cuh -- host-side launch of the decode kernels for one layout,
// dispatching on the GQA group size G = Hq / Hkv (1..8).
#pragma once

#include "decode_attention.cuh"

namespace pkv {

constexpr int kDecodeStages = 3;  // per-warp ring depth (3 x 8 KiB per warp)

// Dynamic shared memory of the main kernel for group size g.
int decode_smem_bytes(int g);

// Sets the kernel's dynamic shared-memory limit once per device.
template <typename Kernel>
cudaError_t ensure_smem_limit(Kernel kernel, int bytes, unsigned long long* done_mask) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (__atomic_load_n(done_mask, __ATOMIC_ACQUIRE) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) __atomic_fetch_or(done_mask, bit, __ATOMIC_ACQ_REL);
  return e;
}

// Clusters of 2, 4, 8 and 16 of the kernel's CTAs that the current device holds
// at once (asked once a device).
struct ClusterRoom {
  int held[4];
};

template <typename Kernel>
cudaError_t cluster_room(Kernel kernel, int threads, int bytes, ClusterRoom (&rooms)[64],
                         unsigned long long* asked, ClusterRoom* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  ClusterRoom& room = rooms[dev & 63];
  if (!(__atomic_load_n(asked, __ATOMIC_ACQUIRE) & bit)) {
    const bool wide =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    for (int i = 0; i < 4; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2u << i);
      cfg.blockDim = dim3(threads);
      cfg.dynamicSmemBytes = bytes;
      cudaLaunchAttribute attr[1] = {};
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2u << i;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int count = 0;
      if ((i == 3 && !wide) ||
          cudaOccupancyMaxActiveClusters(&count, kernel, &cfg) != cudaSuccess)
        count = 0;
      __atomic_store_n(&room.held[i], count, __ATOMIC_RELAXED);
    }
    cudaGetLastError();  // (a size that the device does not have)
    __atomic_fetch_or(asked, bit, __ATOMIC_ACQ_REL);
  }
  for (int i = 0; i < 4; ++i) out->held[i] = __atomic_load_n(&room.held[i], __ATOMIC_RELAXED);
  return cudaSuccess;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(bool pdl, void (*kernel)(KArgs...), dim3 grid, int cluster, size_t smem,
                           cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kDecodeThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <int G, bool kContig, bool kScored>
cudaError_t launch_decode_group(const DecodeParams& p, cudaStream_t stream) {
  using L = DecodeSmemLayout<G, kDecodeStages>;
  static unsigned long long done_mask = 0;
  auto kernel = decode_attention_kernel<G, kContig, kDecodeStages, kScored>;
  cudaError_t e = ensure_smem_limit(kernel, L::kTotal, &done_mask);
  if (e != cudaSuccess) return e;
  // the scored kernels are programmatic dependents (both wait before they
  // read anything): small calls, where a launch's latency counts
  const bool pdl = kScored ? pdl_decode_enabled() : pdl_enabled();
  if constexpr (kScored) {
    if (p.cluster > 0)  // the splits are a cluster that joins them itself
      return launch_cluster(pdl, kernel, dim3(p.cluster, p.Hkv, p.num_seqs), p.cluster, L::kTotal,
                            stream, p);
  }
  const dim3 grid(p.nsplit, p.Hkv, p.num_seqs);
  e = launch_pdl_if(pdl, kernel, grid, dim3(kDecodeThreads), L::kTotal, stream, p);
  if (e != cudaSuccess || p.nsplit == 1) return e;
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.Hq;
  return launch_pdl_if(pdl, decode_combine_kernel<kContig, kScored>,
                       dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, stream, p);
}

template <bool kContig, bool kScored = false>
cudaError_t launch_decode(const DecodeParams& p, int group, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_decode_group<1, kContig, kScored>(p, stream);
    case 2: return launch_decode_group<2, kContig, kScored>(p, stream);
    case 3: return launch_decode_group<3, kContig, kScored>(p, stream);
    case 4: return launch_decode_group<4, kContig, kScored>(p, stream);
    case 5: return launch_decode_group<5, kContig, kScored>(p, stream);
    case 6: return launch_decode_group<6, kContig, kScored>(p, stream);
    case 7: return launch_decode_group<7, kContig, kScored>(p, stream);
    case 8: return launch_decode_group<8, kContig, kScored>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

// The room for clusters of the scored kernel of a group size.
template <int G, bool kContig>
cudaError_t room_of_group(ClusterRoom* out) {
  using L = DecodeSmemLayout<G, kDecodeStages>;
  static unsigned long long done_mask = 0, asked = 0;
  static ClusterRoom rooms[64];
  auto kernel = decode_attention_kernel<G, kContig, kDecodeStages, true>;
  const cudaError_t e = ensure_smem_limit(kernel, L::kTotal, &done_mask);
  return e != cudaSuccess ? e : cluster_room(kernel, kDecodeThreads, L::kTotal, rooms,
                                                 &asked, out);
}

template <bool kContig>
cudaError_t decode_cluster_room(int group, ClusterRoom* out) {
  switch (group) {
    case 1: return room_of_group<1, kContig>(out);
    case 2: return room_of_group<2, kContig>(out);
    case 3: return room_of_group<3, kContig>(out);
    case 4: return room_of_group<4, kContig>(out);
    case 5: return room_of_group<5, kContig>(out);
    case 6: return room_of_group<6, kContig>(out);
    case 7: return room_of_group<7, kContig>(out);
    case 8: return room_of_group<8, kContig>(out);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_decode_paged(const DecodeParams& p, int group, cudaStream_t stream);
cudaError_t launch_decode_contig(const DecodeParams& p, int group, cudaStream_t stream);
// capped, biased and masked scores (p.sp)
cudaError_t launch_decode_paged_scored(const DecodeParams& p, int group, cudaStream_t stream);
cudaError_t launch_decode_contig_scored(const DecodeParams& p, int group, cudaStream_t stream);
cudaError_t room_decode_paged_scored(int group, ClusterRoom* out);
cudaError_t room_decode_contig_scored(int group, ClusterRoom* out);

}  // namespace pkv
