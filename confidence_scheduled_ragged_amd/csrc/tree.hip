// tree.hip - drafted trees: the ancestors of every node, and the walk down a
// tree by the target's choices.
//
// The packed rows of a request are the nodes of a tree (or of several): row j
// has the parent parents[r] among the request's rows, which is below j; any
// other value makes it a root.
#include "forward.hpp"

namespace dspark {

constexpr int kMaskThreads = 256;
constexpr int kWalkThreads = 256;

// The rows [start, start + n) of a request, within the packed arrays.
__device__ __forceinline__ void rows_of(const int32_t *cu, int b, int rows, int max_rows,
                                        int &start, int &n) {
    int s = cu[b], e = cu[b + 1];
    s = s < 0 ? 0 : (s > rows ? rows : s);
    e = e < s ? s : (e > rows ? rows : e);
    start = s;
    n = e - s < max_rows ? e - s : max_rows;
}
__device__ __forceinline__ int parent_of(int parent, int j) {
    return parent >= 0 && parent < j ? parent : -1;
}

// One workgroup per request: its parents lie in LDS, and a thread walks from one
// node to its root for one word of that node's mask. An ancestor `step` levels up
// is in the window when step < window, and among the first positions when
// ctx + depth - step < sinks. The depth is known at the end of the walk, so those
// few rows that need it walk twice. Up to 64 nodes it is bound by its launch and three
// dependent reads: one tree of 32 nodes takes 2.7 us, 192 of up to 64 nodes 4.4. Walks
// beside each other take as many steps as a tree is deep; filling the masks node by node
// would take as many as it has nodes. But each word of a node is a walk of its own, and
// 256 threads share nodes x words of them: one tree of 256 nodes, 10 deep, takes 11 us
// (64 such trees 12), one of 1024 nodes 123, a chain of 256 nodes 99 us and one of 1024
// 5.5 ms (11 with sinks past its window); one walk a node would be a 32nd of these steps.
__global__ __launch_bounds__(kMaskThreads) void tree_masks_kernel(TreeMaskParams p) {
    __shared__ int parent_s[DSPARK_MAX_TREE];
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        int start, n;
        rows_of(p.cu, b, p.rows, p.max_rows, start, n);
        const int ctx = p.ctx ? (p.ctx[b] < 0 ? 0 : p.ctx[b]) : 0;
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += kMaskThreads)
            parent_s[j] = parent_of(p.parents[start + j], j);
        __syncthreads();
        for (int i = threadIdx.x; i < n * p.words; i += kMaskThreads) {
            const int j = i / p.words, w = i - j * p.words;
            uint32_t bits = 0;
            int depth = 0;
            for (int k = j, step = 0; k >= 0; k = parent_s[k], ++step) {
                if (k >> 5 == w && (p.window == 0 || step < p.window)) bits |= 1u << (k & 31);
                depth = step;
            }
            if (p.window > 0 && depth >= p.window && ctx < p.sinks)
                for (int k = j, step = 0; k >= 0; k = parent_s[k], ++step)
                    if (k >> 5 == w && (int64_t)ctx + depth - step < p.sinks)
                        bits |= 1u << (k & 31);
            p.masks[(int64_t)(start + j) * p.words + w] = bits;
            if (w == 0) p.depths[start + j] = depth;
        }
    }
}

// One wave per request. From row 0 on: the lowest row that has the current one
// for its parent and the target's choice there for its token is next. Up to 64
// rows stay in the lanes' registers, so that a level costs no memory access. Bound by
// its launch and two dependent reads: 3.0 us for one tree, 4.9 for 256.
__global__ __launch_bounds__(kWalkThreads) void tree_accept_kernel(TreeAcceptParams p) {
    const int lane = threadIdx.x & (kWave - 1);
    const int b = blockIdx.x * (kWalkThreads / kWave) + threadIdx.x / kWave;
    if (b >= p.B) return;
    int start, n;
    rows_of(p.cu, b, p.rows, p.max_rows, start, n);
    int32_t *path = p.path + (int64_t)b * p.width;
    auto row = [&](int j, int &parent, int &token, int &choice) {
        parent = j < n ? parent_of(p.parents[start + j], j) : -1;
        token = j < n ? p.tokens[start + j] : 0;
        choice = j < n ? p.choice[start + j] : 0;
    };
    int parent, token, choice;
    row(lane, parent, token, choice);
    int at = n > 0 ? 0 : -1, depth = 0, want = -1;
    if (at == 0) {
        want = __shfl(choice, 0, kWave);
        if (lane == 0) path[0] = 0;
    }
    while (at >= 0 && depth + 1 < p.width) {
        int next = -1, then = -1;
        uint64_t child = __ballot(parent == at && token == want);
        if (child) {
            next = __ffsll((unsigned long long)child) - 1;
            then = __shfl(choice, next, kWave);
        }
        for (int j0 = kWave; j0 < n && next < 0; j0 += kWave) {
            int q, t, c;
            row(j0 + lane, q, t, c);
            child = __ballot(q == at && t == want);
            if (!child) continue;
            const int l = __ffsll((unsigned long long)child) - 1;
            next = j0 + l;
            then = __shfl(c, l, kWave);
        }
        if (next < 0) break;
        at = next;
        want = then;
        ++depth;
        if (lane == 0) path[depth] = at;
    }
    for (int i = (at < 0 ? 0 : depth + 1) + lane; i < p.width; i += kWave) path[i] = -1;
    if (lane == 0) {
        p.accepted[b] = depth;
        p.bonus[b] = want;
    }
}

hipError_t launch_tree_masks(const TreeMaskParams &p, hipStream_t s) {
    const int grid = p.B < (1 << 16) ? p.B : 1 << 16;
    hipLaunchKernelGGL(tree_masks_kernel, dim3((unsigned)grid), dim3(kMaskThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_tree_accept(const TreeAcceptParams &p, hipStream_t s) {
    const int per = kWalkThreads / kWave;
    hipLaunchKernelGGL(tree_accept_kernel, dim3((unsigned)((p.B + per - 1) / per)),
                       dim3(kWalkThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace dspark
