// How large the clusters of the recurrence's scans are (host code, without CUDA).
#pragma once

#include <algorithm>

namespace moe {

constexpr int kMaxCluster = 16;  // blocks of a cluster

// How many clusters of each size the GPU has room for at once.
struct ClusterRoom {
  int clusters[kMaxCluster + 1] = {};
};

// ask(c, &n): whether clusters of c blocks can be launched, and how many run at once.  A size that
// cannot is left out; single blocks always can.
template <typename Ask>
ClusterRoom ask_room(Ask ask) {
  ClusterRoom r;
  for (int c = 1; c <= kMaxCluster; ++c) {
    int n = 0;
    r.clusters[c] = ask(c, &n) ? std::max(n, 0) : 0;
  }
  r.clusters[1] = std::max(r.clusters[1], 1);
  return r;
}

struct ClusterChoice {
  int cluster, parts;
};

// As large clusters as can all run at once, up to 8 blocks; where these leave room, sequences are
// parted.  Larger clusters (whose exchanges take longer) only where they put more blocks to work:
// few channels in few sequences (65536 x 64, one sequence: 107 us in clusters of 8, 63 us of 16;
// 65536 x 512, 24 sequences: 51 us of 8 and 89 us of 16).
inline ClusterChoice choose_clusters(const ClusterRoom& room, int strips, int tiles, int n_seq) {
  const auto parts = [&](int c) {
    return std::max(1, std::min({n_seq, tiles, room.clusters[c] / strips}));
  };
  int cluster = 1;
  for (int c = 2; c <= std::min(kMaxCluster, tiles); ++c)
    if (room.clusters[c] >= strips && (c <= 8 || c * parts(c) > cluster * parts(cluster)))
      cluster = c;
  return {cluster, parts(cluster)};
}

}  // namespace moe
