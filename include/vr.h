/*
 * vr.h -- emulated Ring / Double-Binary-Tree AllReduce on one GPU.
 *
 * R "virtual ranks" are R device buffers in one GPU's memory.  The library
 * computes what an AllReduce (ReduceScatter, AllGather) over R ranks
 * computes, following the ring and double-binary-tree schedules, and writes
 * every rank's result buffer.  Each fused collective call is one kernel
 * launch on the caller's stream (the host-buffer and non-fused variants
 * enqueue several); nothing crosses a GPU or process boundary.
 *
 * Sources (web pages), cited below as [tag] "section":
 *   [Course13]  "NCCL 专家课程 13：Tree、双树、层次化连接与真实交叉区间" (blog.cptz.space)
 *   [Internals] "NCCL 内部机制：一次 AllReduce 如何变成拓扑图、Channel 与 GPU Kernel"
 *               (charlestar.github.io)
 *   [CodeNotes] "NCCL代码分析" (jianzi123.github.io)
 *   [Interview] "all-reduce 每张卡要发多少数据? ring 和 tree 有什么区别?"
 *               (charliedreemur.github.io)
 *
 * Conventions shared by every call
 *   - All functions are thread-safe.  They return VR_SUCCESS or an error code;
 *     argument errors are detected on the host before anything is enqueued.
 *   - Buffers are owned by the caller.  The pointer arrays are read during the
 *     call only (their contents are passed to the kernel by value), so the
 *     caller may reuse or free the arrays as soon as the call returns.
 *   - Collective calls are asynchronous on `stream` (a cudaStream_t; NULL is
 *     the legacy default stream): returning means enqueued, not completed
 *     ([Internals] "API 返回只意味着提交边界，不意味着数据已经可读").  Read the
 *     result only after synchronising the stream or through a stream-ordered
 *     dependency.
 *   - The library allocates no device buffers at run time.  Its own device
 *     state is static: one status word and one bounds word per device and
 *     the 8 MiB FIFO of vr_allreduce_ring_stepwise_noalloc (__device__
 *     variables), plus the code
 *     of kernels compiled at run time (vr_jit_status) and, once
 *     vr_allreduce_host has run on a device, two streams and four events
 *     there.  vr_finalize releases what is not static.
 *   - Reductions accumulate in fp32 for every dtype and narrow to the element
 *     type once, round-to-nearest-even.  Sum is IEEE fp32 addition in the
 *     schedule's order; Max returns the larger value, with +0 above -0.
 *   - Results are deterministic: the same call on the same inputs gives the
 *     same bits, and every rank's output is bit-identical.
 *
 * Options, for tests and tuning (no option changes a result, only which
 * kernel computes it, or what the library prints).  Each is read from the
 * environment once, at the first call that needs an option, and changed
 * afterwards only through vr_set_option (same names and values):
 *   VR_KERNEL_PATH=staged|register  force the shared-memory-staged or the
 *                                   register-path AllReduce / ReduceScatter
 *                                   kernel (aligned buffers); vr_set_option
 *                                   takes 2 or 1 (0: automatic)
 *   VR_JIT=0                        interpreting tree / ring folds only
 *   VR_JIT_RING=0|1                 ring folds specialised: never / also on
 *                                   the staged kernel
 *   VR_SMALL_RANKS=0                no few-rank register-path variant
 *   VR_SPREAD=0                     256-thread CTAs even when a small call
 *                                   would leave SMs idle
 *   VR_JIT_OCC=0|4                  specialised register-path kernels at
 *                                   four CTAs per SM: never / always (by
 *                                   default a tree call takes them when
 *                                   each thread folds at most three units
 *                                   and the larger grid saves every thread
 *                                   one)
 *   VR_PDL=0                        launch without programmatic stream
 *                                   serialisation (by default a kernel may
 *                                   start while the previous one on the
 *                                   stream drains; it waits for it before
 *                                   touching memory)
 *   VR_STAGED_MIN_BYTES=n           staged kernel from n bytes per rank
 *                                   (default 16 MiB; 2-7 ranks: from the
 *                                   larger of n and 32 MiB; trees that draw
 *                                   their tiles (VR_SCHED): above 8 ranks
 *                                   from n / 2, 5-7 ranks from the larger
 *                                   of n and 24 MiB)
 *   VR_STAGED_TILE_BYTES, VR_STAGED_STAGES, VR_STAGED_MIN_STAGES
 *                                   staged geometry: bytes per rank per
 *                                   tile, most stages, fewest stages
 *   VR_AG_TILE, VR_AG_STAGES, VR_AG_CTAS
 *                                   TMA AllGather geometry (pairs of tile
 *                                   and stages that are compiled: 8192/4,
 *                                   8192/8, 16384/4, 16384/6, 32768/3,
 *                                   4096/8; others are INVALID_ARGUMENT)
 *   VR_AG_ORDER=1|2                 TMA AllGather tile order: source-major
 *                                   (each loaded tile stored to all R
 *                                   outputs) / destination-major (each
 *                                   output written in long runs, sources
 *                                   re-read from L2); by default
 *                                   destination-major when the R sources
 *                                   take at most a quarter of L2
 *   VR_SCHED=0|1|2                  staged AllReduce: 0 every CTA takes a
 *                                   fixed run of tiles; 1 (default) the
 *                                   CTAs draw tiles at run time where that
 *                                   measured faster (trees of 4 or more
 *                                   ranks, 8 excepted; rings of 16 or
 *                                   more, and fp32 rings of 4 and of 9
 *                                   or more);
 *                                   2 always drawn.
 *                                   Drawing uses a scheduler slot in
 *                                   device memory per stream, and one per
 *                                   launch captured into a graph: launches
 *                                   on one stream, and the replays of one
 *                                   instantiated graph, run one after
 *                                   another.  Two instances of one captured
 *                                   graph running at the same time share
 *                                   the captured launch's slot; the later
 *                                   one's CTAs wait (bounded) and report
 *                                   VR_ERR_TIMEOUT if it stays held (a
 *                                   slot so left held fails later drawing
 *                                   calls on it the same way until
 *                                   vr_debug_sched_slot frees it).
 *                                   Slots per device: 1024 streams and
 *                                   3072 captured launches; past them,
 *                                   fixed runs.  The same bits either way.
 *   VR_DEBUG=GRAPH                  print every tree set, ring and channel
 *                                   partition a call plans to stderr, in
 *                                   the log formats of [Course13] "从 GRAPH
 *                                   日志复原 active tree" (vr_set_option
 *                                   takes 1)
 * Read once at first use, not changeable:
 *   VR_WAIT_TIMEOUT_NS=n            limit of every bounded wait
 *                                   (default 1 s)
 *   VR_VALIDATE_POINTERS=1          check that every buffer is reachable
 *                                   from the current device
 */
#ifndef VR_H
#define VR_H

#ifndef __CUDACC_RTC__
#include <stddef.h>
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  VR_SUCCESS = 0,
  VR_ERR_INVALID_ARGUMENT = 1, /* bad size, pointer, overlap or enum value */
  VR_ERR_UNSUPPORTED = 2,      /* valid arguments, combination not offered  */
  VR_ERR_CUDA = 3,             /* a CUDA runtime call failed                */
  VR_ERR_TIMEOUT = 4,          /* a bounded device-side wait ran out        */
  VR_ERR_INTERNAL = 5          /* a library invariant failed (bounds fault) */
} vr_result_t;

typedef enum { VR_FLOAT32 = 0, VR_FLOAT16 = 1, VR_BFLOAT16 = 2 } vr_dtype_t;
typedef enum { VR_SUM = 0, VR_MAX = 1 } vr_op_t;
/* VR_ALGO_AUTO (AllReduce only): ring or tree, whichever the cost model
 * (vr_select_algo) predicts faster. */
typedef enum { VR_ALGO_RING = 0, VR_ALGO_TREE = 1, VR_ALGO_AUTO = 2 } vr_algo_t;

#define VR_MAX_RANKS 64
#define VR_MAX_CHANNELS 64

/* One rank's view of one tree: the ncclTree record of [Course13]
 * "数据结构不是纯二叉树".  up = parent rank (-1 at the root); down[] = child
 * ranks, present children first, empty slots -1; depth = the approximation
 * localRanks - 1 + floor(log2(nNodes)) of [Course13] "节点间连接". */
typedef struct {
  int depth;
  int up;
  int down[3];
} vr_tree_t;

/* ------------------------------------------------------------ topology */

/* Identity ring of every channel ([Interview] "先弄清楚": each rank sends to
 * its right-hand neighbour).  next[c*R + r] = (r+1) mod R and
 * prev[c*R + r] = (r-1) mod R for c < nChannels.  `next` and `prev` are
 * caller-owned host arrays of nChannels*R ints.
 * Errors: VR_ERR_INVALID_ARGUMENT for R outside [1, VR_MAX_RANKS], nChannels
 * outside [1, VR_MAX_CHANNELS] or a NULL array. */
vr_result_t vr_build_ring(int R, int nChannels, int* next, int* prev);

/* Hierarchical double binary tree over R = nNodes*localRanks ranks
 * ([Course13] "节点内先形成链", "节点间连接", "Btree 的 bit 构造",
 * "双树：偶数 mirror，奇数 shift").  Within a node the ranks k*L .. k*L+L-1
 * form a chain (up = previous, down[0] = next).  Over node indices, tree 0 is
 * the bit-trick binary tree and tree 1 its mirror (even nNodes) or its
 * one-step shift (odd nNodes); the head k*L of node k takes up = head of its
 * parent node and appends the heads of its child nodes to down[].
 * Channels [0, ceil(nChannels/2)) carry tree 0, the others tree 1.
 * `trees` is a caller-owned host array of nChannels*R records,
 * trees[c*R + r].  localRanks = 1 gives the flat double binary tree.
 * Errors: VR_ERR_INVALID_ARGUMENT for R outside [1, VR_MAX_RANKS], nNodes or
 * localRanks < 1, nChannels outside [1, VR_MAX_CHANNELS], NULL `trees`. */
vr_result_t vr_build_dtree(int nNodes, int localRanks, int nChannels, vr_tree_t* trees);

/* Which rank of a node's intra order joins the node-level tree
 * ([Course13] "节点内先形成链"): the parent head is always the first; the
 * heads that take child nodes d0 / d1 are the first / first (TREE), the
 * second / second (SPLIT_TREE) or the second / first (BALANCED_TREE). */
typedef enum {
  VR_PATTERN_TREE = 0,
  VR_PATTERN_SPLIT_TREE = 1,
  VR_PATTERN_BALANCED_TREE = 2
} vr_tree_pattern_t;

/* vr_build_dtree with a head pattern and per-channel intra-node orders
 * ([Course13] "节点内先形成链": the chain follows treeIntra, which a topology
 * search may order differently per channel; "本机真实树形" shows such
 * channels).  intraOrders: NULL (identity) or nChannels*localRanks ints, row
 * c a permutation of 0..localRanks-1 giving channel c's chain order inside
 * every node.  The parent head of node k takes up = the child0 or child1
 * head of its parent node (by k's parentChildType in the node-level tree);
 * the child0 head appends child node d0's parent head, then the child1 head
 * appends d1's.  Errors: those of vr_build_dtree, plus
 * VR_ERR_INVALID_ARGUMENT for a bad pattern, SPLIT_TREE / BALANCED_TREE
 * with one local rank, or a row that is not a permutation. */
vr_result_t vr_build_dtree_ex(int nNodes, int localRanks, int nChannels,
                              vr_tree_pattern_t pattern, const int* intraOrders,
                              vr_tree_t* trees);

/* Channel c's element range of a message of `count` elements ([Course13]
 * "前置知识": channels take different ranges of one message).  The message
 * is cut into 16-byte grains, split over channels so that the first
 * (grains mod nChannels) channels get one more grain, and clipped at count.
 * Writes *offset and *channelCount (elements).
 * Errors: VR_ERR_INVALID_ARGUMENT for a bad dtype, nChannels outside
 * [1, VR_MAX_CHANNELS], channel outside [0, nChannels) or NULL outputs. */
vr_result_t vr_partition(size_t count, vr_dtype_t dtype, int nChannels, int channel,
                         size_t* offset, size_t* channelCount);

/* Ring block of element `elem` in the ring AllReduce partition, which fixes
 * the order in which the element is reduced ([Interview] "手撕代码": the
 * block leaves rank j first and each later rank adds its copy).  A channel is
 * walked in loops of R*C elements (C = chunkBytes / element size), the last
 * loop shorter; each loop is cut into R blocks, the first (loop mod R) one
 * element longer.  Writes *channel and *block (the block number j).
 * Errors: VR_ERR_INVALID_ARGUMENT for elem >= count or the argument errors
 * of vr_allreduce. */
vr_result_t vr_ring_block(size_t count, vr_dtype_t dtype, int R, int nChannels,
                          size_t chunkBytes, size_t elem, int* channel, int* block);

/* --------------------------------------------------------- collectives */

/* AllReduce: every recvbufs[r] (count elements) receives the reduction over
 * r' < R of sendbufs[r'] ([Internals] "从 API 调用到可调度任务": two buffers,
 * count, dtype, op, communicator and stream).
 *   RING ([Interview] "手撕代码", [Internals] "Ring：带宽友好"): an element in
 *        block j of its ring loop is reduced over ranks j, j+1, ..., j+R-1
 *        (mod R), left to right -- reduce-scatter followed by all-gather.
 *   TREE ([Course13] "先固定方向", "runTreeSplit 如何流水", "每种 rank 的操作"):
 *        on the channel's tree every rank folds its local input with its
 *        children's partials in down[] order and passes the result up; the
 *        root's value is broadcast down to all ranks.  localRanks = 1 here.
 *   AUTO the one of the two that vr_select_algo predicts faster.
 * nChannels in [1, VR_MAX_CHANNELS] splits the message (vr_partition);
 * chunkBytes (a positive multiple of 16) is the per-rank chunk C of a ring
 * loop and the chunk of a tree channel.
 * In place: sendbufs[r] == recvbufs[r] is allowed.
 * Buffers: any alignment.  16-byte aligned buffers run 16-byte units: from
 * 16 MiB per rank the ring and the tree with 8..64 ranks (the tree with
 * 9..64 ranks from 8 MiB), and from 32 MiB per rank those with 2..7 ranks
 * (the tree with 5..7 from 24 MiB; not the ring of 6), run on a kernel that
 * stages each tile of all R ranks in shared memory with bulk asynchronous
 * copies (the tree's fold specialised at run time, see vr_jit_status),
 * everything else on a kernel that loads the ranks' units into registers
 * (rings of at most 64 Ki elements per rank: one element per thread).  The
 * ring of two ranks runs the tree kernels (two operands fold to the same bits
 * in either order).  The option VR_KERNEL_PATH (staged|register; see the top
 * of this header) forces one of the two for testing and tuning; results are
 * identical.  Unaligned buffers run element units on the register kernel.
 * Errors (nothing enqueued): VR_ERR_INVALID_ARGUMENT for R outside
 * [1, VR_MAX_RANKS], NULL arrays, a NULL buffer with count > 0, a buffer not
 * aligned to the element size, a bad enum, bad nChannels or chunkBytes, or a
 * recv buffer that overlaps another rank's send or recv buffer or partly
 * overlaps its own send buffer.
 * count == 0 enqueues nothing.  R == 1 copies (or leaves in place). */
vr_result_t vr_allreduce(const void* const* sendbufs, void* const* recvbufs, int R,
                         size_t count, vr_dtype_t dtype, vr_op_t op, vr_algo_t algo,
                         int nChannels, size_t chunkBytes, void* stream);

/* vr_allreduce with a hierarchical rank layout: R = nNodes * localRanks,
 * node k holding ranks k*localRanks .. (k+1)*localRanks - 1.  TREE uses the
 * trees of vr_build_dtree(R / localRanks, localRanks, nChannels); RING is the
 * same as vr_allreduce.  Extra error: localRanks < 1 or not dividing R. */
vr_result_t vr_allreduce_ex(const void* const* sendbufs, void* const* recvbufs, int R,
                            size_t count, vr_dtype_t dtype, vr_op_t op, vr_algo_t algo,
                            int nChannels, size_t chunkBytes, int localRanks, void* stream);

/* vr_allreduce_ex on HOST buffers, pipelined through a device workspace.
 * [Internals] "API 返回只意味着提交边界": the call enqueues and returns; here
 * the enqueued work also moves the data in and out.  The message is cut into
 * pieces of pieceBytes per rank (0: VR_HOST_PIECE_BYTES; else a multiple of
 * 16).  Piece p is copied in to workbufs on one internal stream, folded in
 * place there on `stream`, and copied out to recvbufs on another internal
 * stream, so copies in both directions overlap the fold of other pieces.
 * The result equals vr_allreduce_ex's bit for bit: an element's fold reads
 * only that element of each rank, in the order the whole message's
 * partition gives it.
 *   sendbufs[r], recvbufs[r]: host memory, count elements; page-locked for
 *     the copies to overlap (pageable memory works, serialised); in place
 *     (recvbufs[r] == sendbufs[r]) allowed.  They must stay valid, and
 *     sendbufs unchanged, until `stream` has passed this call.
 *     recvbufs[r] may be NULL: rank r's result is then not copied out and
 *     stays in workbufs[r] only (every rank's result is the same vector, so
 *     a caller that needs one copy on the host names one receive buffer).
 *   workbufs[r]: device memory of the current device, count elements each,
 *     owned by the caller; overwritten.
 *   stream: nothing is copied in before the caller's earlier work on it is
 *     done, and work the caller enqueues on it after this call waits for the
 *     last copy out.
 * The internal streams and events are created per device on first use and
 * destroyed by vr_finalize.  Calls from several threads are serialised on
 * the host.  Errors as vr_allreduce_ex, plus VR_ERR_INVALID_ARGUMENT for a
 * NULL workbufs, a pieceBytes not a multiple of 16, a workspace buffer that
 * is not device memory of the current device, or a host buffer that is
 * device memory. */
#define VR_HOST_PIECE_BYTES ((size_t)8 << 20)
vr_result_t vr_allreduce_host(const void* const* sendbufs, void* const* recvbufs, int R,
                              size_t count, vr_dtype_t dtype, vr_op_t op, vr_algo_t algo,
                              int nChannels, size_t chunkBytes, int localRanks,
                              void* const* workbufs, size_t pieceBytes, void* stream);

/* Tree AllReduce over caller-given trees: channel c folds every element over
 * trees[c*R .. c*R + R-1] (vr_tree_t records, e.g. from vr_build_dtree_ex)
 * in the order of vr_allreduce's TREE: each rank folds its local input with
 * its children's partials in down[] order, the root's value goes to every
 * rank.  Each channel's records must form one tree over the R ranks: up and
 * down[] agree both ways, down[] has its present children first, one root,
 * every rank reaches it.  At most 16 distinct trees per call.  Host-side
 * errors: those of vr_allreduce, VR_ERR_INVALID_ARGUMENT for a NULL or
 * invalid tree, VR_ERR_UNSUPPORTED for more than 16 distinct trees or a tree
 * whose fold keeps more than 8 partials live. */
vr_result_t vr_allreduce_trees(const void* const* sendbufs, void* const* recvbufs, int R,
                               size_t count, vr_dtype_t dtype, vr_op_t op, int nChannels,
                               size_t chunkBytes, const vr_tree_t* trees, void* stream);

/* ReduceScatter ([Interview] "先弄清楚": each rank keeps the reduced 1/n
 * segment it is responsible for): sendbufs[r] holds R*recvcount elements;
 * recvbufs[b] (recvcount elements) receives block b = elements
 * [b*recvcount, (b+1)*recvcount) reduced over all ranks, in ring order
 * b+1, b+2, ..., b (mod R).  Only VR_ALGO_RING: tree implements AllReduce
 * only ([CodeNotes] "通讯时如何选择Channel"), so VR_ALGO_TREE returns
 * VR_ERR_UNSUPPORTED.  In place: recvbufs[r] == sendbufs[r] + r*recvcount
 * (in elements).  fp32 with 2..8 ranks from 16 MiB sent per rank runs the
 * shared-memory-staged kernel (64 KB stages), everything else the register
 * kernel.  Other errors as vr_allreduce. */
vr_result_t vr_reduce_scatter(const void* const* sendbufs, void* const* recvbufs, int R,
                              size_t recvcount, vr_dtype_t dtype, vr_op_t op,
                              vr_algo_t algo, int nChannels, size_t chunkBytes,
                              void* stream);

/* AllGather ([Interview] "先弄清楚": the segments are concatenated back):
 * recvbufs[q] (R*sendcount elements) receives sendbufs[r] (sendcount
 * elements) at elements [r*sendcount, (r+1)*sendcount) for every r -- an exact
 * copy.  Only VR_ALGO_RING (VR_ALGO_TREE: VR_ERR_UNSUPPORTED).  In place:
 * sendbufs[r] == recvbufs[r] + r*sendcount.  Other errors as vr_allreduce. */
vr_result_t vr_allgather(const void* const* sendbufs, void* const* recvbufs, int R,
                         size_t sendcount, vr_dtype_t dtype, vr_algo_t algo,
                         int nChannels, size_t chunkBytes, void* stream);

/* ------------------------------------------------ non-fused variants
 * Same results as the fused calls above, computed the way a schedule that
 * moves messages between ranks does, to measure what fusion buys. */

/* Two-phase tree AllReduce ([Course13] "当前环境命中哪个 device 实现":
 * runTreeUpDown reduces the whole message up the tree before broadcasting it
 * down; runTreeSplit overlaps the two).  First launch: every unit is folded
 * over its channel's tree and stored to the tree root's receive buffer only;
 * second launch: copied from there to every other rank.  Same arguments,
 * errors and bits as vr_allreduce_ex with VR_ALGO_TREE; one more read and
 * write of the message.  Two kernel launches. */
vr_result_t vr_allreduce_tree_updown(const void* const* sendbufs, void* const* recvbufs, int R,
                                     size_t count, vr_dtype_t dtype, vr_op_t op, int nChannels,
                                     size_t chunkBytes, int localRanks, void* stream);

/* Bytes of device scratch vr_allreduce_ring_stepwise needs: count elements
 * of dtype, rounded up to 16 (0 for a bad dtype). */
size_t vr_ring_stepwise_scratch_bytes(size_t count, vr_dtype_t dtype);

/* Stepwise ring AllReduce ([Interview] "手撕代码"; [Internals] "Ring：带宽友好"):
 * the ring's 2(R-1) steps run one after the other, each as two launches, and
 * every message crosses device memory: each step first copies every rank's
 * outgoing block (of every loop) into the caller's scratch FIFO, then folds
 * the FIFO into the receiving rank's block (reduce-scatter half) or
 * overwrites it (all-gather half).  recvbufs[r] is rank r's working copy
 * (first set to sendbufs[r]) and keeps partials in the element type, so
 * 16-bit partials are rounded (RNE) at every hop, as messages that travel in
 * that type are; for fp32 and for Max the bits equal vr_allreduce's RING.
 * `scratch` is caller-owned device memory of at least
 * vr_ring_stepwise_scratch_bytes(count, dtype) bytes, aligned to the element
 * size, that overlaps no buffer; its contents are overwritten.  Launches 1 + 4(R-1) kernels.
 * Errors: those of vr_allreduce, plus VR_ERR_INVALID_ARGUMENT for a NULL,
 * short, misaligned or overlapping scratch. */
vr_result_t vr_allreduce_ring_stepwise(const void* const* sendbufs, void* const* recvbufs, int R,
                                       size_t count, vr_dtype_t dtype, vr_op_t op,
                                       int nChannels, size_t chunkBytes, void* scratch,
                                       size_t scratchBytes, void* stream);

/* Size of the device array that vr_allreduce_ring_stepwise_noalloc uses as
 * its message FIFO: 8 MiB per GPU that loads the library. */
#define VR_NOALLOC_SCRATCH_BYTES (8u << 20)

/* vr_allreduce_ring_stepwise for callers that cannot allocate device memory
 * (no counterpart in the pages: it exists for the callers, not the method).
 * A runtime that has given all of the GPU's memory to its own allocator, or
 * code on a latency-critical path that may not call cudaMalloc / cudaFree
 * (both can synchronise the device), cannot supply the scratch FIFO; this
 * entry point uses a file-scope device array of VR_NOALLOC_SCRATCH_BYTES
 * bytes instead, which every GPU that loads the library holds until the
 * process exits.  It allocates nothing, and calls neither cudaMalloc nor
 * cudaFree nor any allocating library routine.
 * Arguments, results and errors are those of vr_allreduce_ring_stepwise
 * without scratch/scratchBytes, plus VR_ERR_UNSUPPORTED when count elements
 * of dtype exceed VR_NOALLOC_SCRATCH_BYTES (2 Mi fp32 or 4 Mi 16-bit
 * elements per rank at most).
 * Arguments are checked first (VR_ERR_INVALID_ARGUMENT as for the other
 * entry point), the size limit after them.
 * Set-up: the first call on a device looks up the array's device address on
 * that device (the device current at the call).  CUDA loads modules lazily,
 * so that first call is also when the device's copy of the array is
 * created: make it before any stream capture, and before the caller's own
 * allocator takes the device's memory (else it can fail with
 * VR_ERR_CUDA).  A call with count == 0 does nothing, set-up included.
 * Sharing: every call on a device uses the same array, which keeps the last
 * call's contents; nothing in it needs to start at zero (each step writes
 * every message before it is read).  Calls whose executions overlap on the
 * GPU (different streams, or different host threads) race on the array:
 * order them. */
vr_result_t vr_allreduce_ring_stepwise_noalloc(const void* const* sendbufs, void* const* recvbufs,
                                               int R, size_t count, vr_dtype_t dtype, vr_op_t op,
                                               int nChannels, size_t chunkBytes, void* stream);

/* ------------------------------------------- operators of a training step
 * What stands directly before and after the AllReduce of a data-parallel
 * step: the losses whose gradients it sums, and the update made of the sum.
 * The pages stop at the collective; these have no counterpart there.  The
 * conventions at the top of this header hold: asynchronous on `stream`,
 * arguments checked before anything is enqueued, no device memory allocated
 * (a call that needs memory takes a workspace of the caller's, at least as
 * large as its ..._workspace_bytes says and 16-byte aligned, whose contents need
 * no initial value and are overwritten; calls that run at the same time need
 * one each), the same bits on every run.  A written buffer may overlap no
 * other buffer of the call unless stated. */

/* Softmax cross entropy of a linear layer over a large vocabulary, with its
 * gradients, without the tokens x vocab logits ever being stored.
 *   l_tv = hidden_t . weight_v,  lse[t] = log sum_v exp l_tv,
 *   losses[t] = lse[t] - l_t,targets[t]  (0 for a token that does not count)
 *   *loss = s * sum_t losses[t],  s = mean ? 1 / (tokens that count) : 1
 *   dHidden = gradScale * d*loss/dhidden,  dWeight = gradScale * d*loss/dweight
 * hidden: `tokens` rows of dim elements, hiddenStride elements apart; weight:
 * `vocab` rows of dim, weightStride apart; both fp16 or both bf16.  targets:
 * 64-bit indices below vocab; ignoreIndex marks a token that does not count
 * (its gradient is zero whatever its hidden state holds).  Any other index
 * outside the vocabulary is ignored too and reported by vr_stream_status as
 * VR_ERR_INVALID_ARGUMENT.  losses, lse: `tokens` floats; loss: one float.
 * dHidden (tokens x dim), dWeight (vocab x dim): contiguous, of dtype; each
 * may be NULL, both for the loss alone.
 * Products are exact and summed in fp32, as are the softmax and the losses;
 * (a confident token's loss is as exact as its logits); in the gradients
 * softmax minus one-hot is rounded to dtype (once, where the numerators are
 * kept twice; fp16: scaled by 2^14 first) and each gradient once (fp16: scale
 * it into range with gradScale).  When no token counts, the loss and the
 * gradients are 0.
 * With gradients, and tokens <= dim (or at most 256 MB of them), the softmax
 * numerators are kept in 16 bits between the passes, if the workspace has
 * room: 6 tokens dim vocab operations.  Else the vocabulary is taken in
 * pieces and the logits are computed twice, 8 tokens dim vocab operations.
 * vr_linear_xent_workspace_bytes gives the size for the loss alone (grads =
 * 0), for the gradients (1), and the least for the gradients (2: in pieces,
 * where that takes less).
 * Rows that are not 16-byte units (dim or stride not a multiple of 8, or a
 * misaligned buffer) are copied into the workspace first; its size depends
 * on the buffers' alignment, so vr_linear_xent_workspace_bytes takes the
 * call's own pointers and strides.
 * Errors: VR_ERR_INVALID_ARGUMENT for fp32 or a bad dtype, dim or vocab < 1,
 * tokens or vocab above 2^30, dim above 2^24, a stride below dim or above
 * 2^32, a NULL or misaligned buffer, an overlap or a short workspace. */
vr_result_t vr_linear_xent_workspace_bytes(const void* hidden, size_t hiddenStride,
                                           const void* weight, size_t weightStride, size_t tokens,
                                           size_t dim, size_t vocab, vr_dtype_t dtype, int grads,
                                           size_t* bytes);
vr_result_t vr_linear_xent(const void* hidden, size_t hiddenStride, const void* weight,
                           size_t weightStride, const long long* targets, size_t tokens,
                           size_t dim, size_t vocab, vr_dtype_t dtype, long long ignoreIndex,
                           int mean, float gradScale, float* losses, float* lse, float* loss,
                           void* dHidden, void* dWeight, void* workspace, size_t workspaceBytes,
                           void* stream);

/* Balance loss of R ranks' expert routers over the whole batch, with its
 * gradients.  logits[r]: `tokens` rows of `experts` router logits (fp32,
 * fp16 or bf16), rowStride elements apart.  Over the N valid tokens of all
 * ranks, with p_t the softmax of a token's logits and c_e the number of
 * tokens whose topK largest logits include expert e (equal logits: the lower
 * expert first; NaN above +inf):
 *   f_e = c_e / (N topK),  P_e = sum_t p_te / N,
 *   *loss = coef * experts * sum_e f_e P_e
 *   dlogits_te = gradScale * coef * experts / N * p_te (f_e - sum_j f_j p_tj)
 * f is held constant in the gradient (the choice has none).
 *   masks: NULL, or R pointers (each may be NULL: every token counts) to
 *     `tokens` bytes, 0 where a token does not count.  A token whose logits
 *     are all -inf does not count either.  Such tokens choose -1 and get a
 *     gradient of zero whatever their logits hold.  A NaN or +inf logit of
 *     a token that counts makes the loss NaN.
 *   counts: `experts` ints, c_e.  loss: one float.
 *   chosen: NULL, or R pointers (each may be NULL) to tokens * topK ints:
 *     each token's experts, the largest logit first.
 *   dlogits: NULL (no gradients), or R buffers laid out as the logits;
 *     dlogits[r] may be logits[r].  Elements between rows are not touched.
 * Softmax and sums are fp32; the gradient is rounded once to dtype (fp16:
 * scale it into range with gradScale).  N = 0 gives loss 0, counts 0.
 * Errors: VR_ERR_INVALID_ARGUMENT for R outside [1, VR_MAX_RANKS], experts
 * outside [1, 1024], topK outside [1, min(experts, 32)], rowStride <
 * experts, R * tokens above 2^31 - 1, a NULL or misaligned buffer, a bad
 * overlap or a short workspace. */
vr_result_t vr_balance_loss_workspace_bytes(int R, size_t tokens, int experts, size_t* bytes);
vr_result_t vr_balance_loss(const void* const* logits, size_t rowStride,
                            const unsigned char* const* masks, int R, size_t tokens, int experts,
                            int topK, vr_dtype_t dtype, float coef, float gradScale, float* loss,
                            int* counts, int* const* chosen, void* const* dlogits,
                            void* workspace, size_t workspaceBytes, void* stream);

/* Matrices of one shape orthogonalised by Newton-Schulz steps, the update an
 * optimiser makes of summed gradients: with X = src / (|src|_F + eps),
 * transposed when rows > cols,
 *   steps times: A = X X^T, X <- a X + (b A + c A A) X
 * and dst = scale * X (transposed back).  Each matrix by itself.
 * src, dst: `count` pointers to contiguous rows x cols matrices of dtype;
 * dst[i] may be src[i].  coefs: NULL (3.4445, -4.775, 2.0315 in every step) or
 * 3 * steps floats on the host, a, b, c of each step.
 * The norm is an fp32 sum of squares (entries beyond about 1e18 overflow
 * it, those below about 1e-19 are lost in it); a zero matrix gives zeros (with
 * eps = 0: NaN), NaN or an infinity a matrix of NaN.  Products are summed in
 * fp32; X is held to 22 bits between the steps, and to 2^-37 where |src|_F far
 * below eps leaves it small.  fp16 and fp32 results, and bf16 results of up to
 * 16 rows or columns, take products of operands of 22 bits (up to three times
 * the time), other bf16 results of operands rounded to 11 bits: an error of
 * the size of the result's own rounding (1e-3 to 3e-3, 2-norm), more where all
 * but a few singular values are zero (up to 1.6e-2 measured with two left).
 * Errors: VR_ERR_INVALID_ARGUMENT for count < 1, rows or cols outside
 * [1, 2^24], steps outside [1, 32], eps negative, or eps, scale or a
 * coefficient not finite, a NULL or misaligned buffer, an overlap or a short
 * workspace; VR_ERR_UNSUPPORTED for coefficients under which singular values
 * starting in [0, 1] can leave the range the operands hold (|X|, |X X^T| and
 * |b A + c A A| up to 15). */
vr_result_t vr_orthogonalize_workspace_bytes(int count, size_t rows, size_t cols,
                                             vr_dtype_t dtype, size_t* bytes);
vr_result_t vr_orthogonalize(const void* const* src, void* const* dst, int count, size_t rows,
                             size_t cols, vr_dtype_t dtype, int steps, const float* coefs,
                             float eps, float scale, void* workspace, size_t workspaceBytes,
                             void* stream);

/* Rows of an embedding table by token, scaled:
 *   out_t = scale * weight_ids[t]
 * rounded once to dtype (fp32, fp16 or bf16).  weight: `vocab` rows of dim
 * elements, weightStride apart; out: `tokens` rows, outStride apart.  ids:
 * 64-bit indices below vocab; a token with ignoreIndex gets a row of zeros, as
 * does one with any other index outside the vocabulary, which vr_stream_status
 * reports as VR_ERR_INVALID_ARGUMENT.  tokens == 0 enqueues nothing.
 * Errors: VR_ERR_INVALID_ARGUMENT for a bad dtype, dim or vocab < 1, tokens or
 * vocab above 2^30, dim above 2^24, a stride below dim or above 2^31, a NULL
 * or misaligned buffer or an overlap. */
vr_result_t vr_embedding(const void* weight, size_t weightStride, const long long* ids,
                         size_t tokens, size_t dim, size_t vocab, vr_dtype_t dtype,
                         long long ignoreIndex, float scale, void* out, size_t outStride,
                         void* stream);

/* The gradient of the table:
 *   dWeight_v = scale * sum_{t: ids[t] = v} dOut_t          (accumulate = 0)
 *   dWeight_v = dWeight_v + scale * sum ...                  (accumulate = 1)
 * dOut: `tokens` rows of dim elements, dOutStride apart; dWeight (vocab x
 * dim): contiguous; both of dtype.  Without accumulate every row is written,
 * zeros for words that do not occur; with it their rows are neither read nor
 * written (the gradient of an output layer that shares the table goes first).
 * Sums are fp32 in token order (many equal tokens: in runs of them, by the numbers
 * of tokens and columns), rounded once to dtype.  Ignored tokens and indices outside
 * the vocabulary as above; what their rows of dOut hold is not read.
 * Errors: those of vr_embedding, or a short workspace. */
vr_result_t vr_embedding_grad_workspace_bytes(size_t tokens, size_t dim, size_t vocab,
                                              vr_dtype_t dtype, size_t* bytes);
vr_result_t vr_embedding_grad(const void* dOut, size_t dOutStride, const long long* ids,
                              size_t tokens, size_t dim, size_t vocab, vr_dtype_t dtype,
                              long long ignoreIndex, float scale, int accumulate, void* dWeight,
                              void* workspace, size_t workspaceBytes, void* stream);

/* Matrix products grouped by expert: rows sorted by group, each times its
 * group's weight.
 *   out_r = weight_e x_r    for the rows r of group e
 * x: `rows` rows of dim elements, xStride apart; weight: `groups` contiguous
 * matrices of outDim rows of dim; out: rows of outDim, outStride apart; all
 * fp16 or all bf16.  counts: `groups` ints on the device, the rows of each
 * group, which follow one another (the counts that vr_balance_loss gives).
 * Any group may have none.  Rows behind the last group's are not read into any
 * result, and their results are left as they were.  Counts that are negative
 * or add up to more than `rows` are cut off there and reported by
 * vr_stream_status as VR_ERR_INVALID_ARGUMENT.
 * Products are exact and summed in fp32 by the tensor cores, which truncate: the
 * longest sums of one piece (32768 terms in fp16, 262144 in bf16; longer ones are
 * taken in chunks) are off by about 3.3e-5 and 2.6e-4 of the running sum, a fifteenth
 * of the result's rounding.  Results are rounded once.  The kernels are chosen by rows / groups: up to 32 rows a group on
 * average are fastest where few have many more (8 of 64 groups with 240 rows each
 * take twice as long as in a buffer of more rows).
 * Rows that are not 16-byte units (dim or stride not a multiple of 8, or a
 * misaligned buffer) are copied into the workspace first, so that its size
 * depends on the call's own pointers and strides.
 * Errors: VR_ERR_INVALID_ARGUMENT for fp32 or a bad dtype, dim or outDim
 * outside [1, 2^24], rows above 2^30, groups outside [1, 1024], a stride below
 * its row or above 2^31, a NULL or misaligned buffer, an overlap or a short
 * workspace. */
vr_result_t vr_grouped_linear_workspace_bytes(const void* x, size_t xStride, const void* weight,
                                              size_t rows, size_t dim, size_t outDim, int groups,
                                              vr_dtype_t dtype, size_t* bytes);
vr_result_t vr_grouped_linear(const void* x, size_t xStride, const void* weight, const int* counts,
                              size_t rows, size_t dim, size_t outDim, int groups, vr_dtype_t dtype,
                              void* out, size_t outStride, void* workspace, size_t workspaceBytes,
                              void* stream);

/* The gradients of such a product:
 *   dX_r = weight_e^T dOut_r,   dWeight_e = sum_{r of group e} dOut_r x_r^T
 * dOut: `rows` rows of outDim elements, dOutStride apart; dX (rows x dim) and
 * dWeight (groups x outDim x dim): contiguous, of dtype; either may be NULL
 * (dX NULL: weight is not used; dWeight NULL: x is not used).  Every
 * group's dWeight is written, zeros for one without rows; rows of dX behind the
 * last group's are left as they were.  Each gradient is rounded once (fp16:
 * scale dOut so that it stays in range).  Otherwise as vr_grouped_linear. */
vr_result_t vr_grouped_linear_grad_workspace_bytes(const void* dOut, size_t dOutStride,
                                                   const void* x, size_t xStride,
                                                   const void* weight, size_t rows, size_t dim,
                                                   size_t outDim, int groups, vr_dtype_t dtype,
                                                   size_t* bytes);
vr_result_t vr_grouped_linear_grad(const void* dOut, size_t dOutStride, const void* x,
                                   size_t xStride, const void* weight, const int* counts,
                                   size_t rows, size_t dim, size_t outDim, int groups,
                                   vr_dtype_t dtype, void* dX, void* dWeight, void* workspace,
                                   size_t workspaceBytes, void* stream);

/* One AdamW step over many tensors at once, in place: with t = step and
 * g = gradScale * grads[i],
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   p = (1 - lr weightDecay) p
 *       - lr / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps)
 * params[i], grads[i], m[i], v[i]: sizes[i] elements (0: skipped), of dtype and
 * gradDtype; any alignment (two to three times as fast where each begins at a
 * multiple of 8 elements).
 *   masters: NULL, or fp32 copies of 16-bit parameters: p is read from and
 *     written to them, and params[i] receives it rounded, unread.
 *   stateBits 32: m, v are fp32 (mScales, vScales NULL).  stateBits 8: m, v are
 *     bytes, and mScales[i], vScales[i] ceil(sizes[i] / 256) floats, one for 256
 *     consecutive elements.  Zeroed bytes and scales are states of zero.  A
 *     byte of m is a sign, four bits of exponent and three of mantissa (the
 *     e4m3 format), one of v five and three, with exponents offset by 15; the
 *     value is that times the block's scale, a power of two by which the block's
 *     largest value begins at 2^7 (m) or 2^15 (v).  New states are rounded at
 *     random, so that they are right on average (a mean over thousands of steps
 *     would stand still otherwise): up or down in proportion to the rest, by 16
 *     random bits that are a function of seed, step and the element's place
 *     among the call's tensors.  A positive v keeps a code above 0.  p is made of the
 *     states before that rounding.  A NaN or an infinity in a block makes its
 *     scale NaN; finite states stay finite (none is rounded up to 2^128).
 *   control: NULL, or three floats in device memory, read when the kernel runs:
 *     lr, step (1 or more) and gradScale in place of the arguments, which a
 *     captured step needs.  A gradScale there that is not finite leaves
 *     everything as it was.
 * States are fp32 operations each rounded by itself, in the order written, with
 * 1 - beta in fp32: the same bits wherever they are computed.
 * The parameter is rounded once: its decay and its move are added first.
 * With eps = 0 an element that never had a gradient becomes NaN (0 / 0).
 * Errors: VR_ERR_INVALID_ARGUMENT for count < 1, a bad dtype, gradDtype or
 * stateBits, masters with fp32 parameters, scales that do not go with
 * stateBits, a size above 2^40, beta1 or beta2 outside [0, 1), eps negative,
 * denormal or not finite, weightDecay or (without control) lr or gradScale not finite or
 * step < 1, a NULL or misaligned buffer, or any overlap. */
vr_result_t vr_adamw(void* const* params, const void* const* grads, void* const* m,
                     void* const* v, float* const* mScales, float* const* vScales,
                     float* const* masters, const size_t* sizes, int count, vr_dtype_t dtype,
                     vr_dtype_t gradDtype, int stateBits, float lr, float beta1, float beta2,
                     float eps, float weightDecay, long long step, float gradScale,
                     unsigned long long seed, const float* control, void* stream);

/* The values of 8-bit states of vr_adamw in fp32, exactly (to look at, or to
 * store in a checkpoint): mValues[i], vValues[i] receive sizes[i] floats;
 * mValues (with m, mScales) or vValues (with v, vScales) may be NULL.
 * Errors: VR_ERR_INVALID_ARGUMENT for count < 1, both NULL, a size above 2^40,
 * a NULL or misaligned buffer, or an overlap. */
vr_result_t vr_adamw_values(const void* const* m, const void* const* v,
                            const float* const* mScales, const float* const* vScales,
                            const size_t* sizes, int count, float* const* mValues,
                            float* const* vValues, void* stream);

/* ---------------------------------------------------------- cost model
 * The pages' alpha-beta model ([Course13] "理想成本模型"; [Interview]
 * "推导 / 关键公式"), with N ranks, tree depth D (the deeper of the two
 * trees, edges from root to deepest leaf) and M bytes per rank:
 *   T_ring = 2(N-1) * alpha[0] + 2(N-1)/N * M * usPerByte[0]
 *   T_tree = 2D     * alpha[1] + 2 M       * usPerByte[1]
 * in microseconds.  The built-in model is fitted (least squares of relative
 * error) to the ring and tree times this library measures on GB300 for
 * 4 ranks, 8 B .. 256 MiB per rank. */
typedef struct {
  double alphaUs[2];    /* per dependent stage: [0] ring, [1] tree */
  double usPerByte[2];  /* per byte of the traffic term: [0] ring, [1] tree */
} vr_cost_model_t;

/* Predicted time of an AllReduce (algo RING or TREE) over R ranks in nodes of
 * localRanks, bytesPerRank each, under `model` (NULL: the current model).
 * Errors: VR_ERR_INVALID_ARGUMENT for a bad algo, R, localRanks or NULL us. */
vr_result_t vr_predict_us(vr_algo_t algo, int R, int localRanks, size_t bytesPerRank,
                          const vr_cost_model_t* model, double* us);

/* The algorithm with the smaller prediction (RING on a tie); what
 * VR_ALGO_AUTO uses with model NULL.  Errors as vr_predict_us. */
vr_result_t vr_select_algo(int R, int localRanks, size_t bytesPerRank,
                           const vr_cost_model_t* model, vr_algo_t* algo);

/* Fits the model to measured AllReduce times: sample i ran R[i] ranks in
 * nodes of localRanks[i], bytesPerRank[i] each, in ringUs[i] and treeUs[i]
 * microseconds (a value <= 0 leaves that algorithm's sample out).  For each
 * algorithm, (alphaUs, usPerByte) minimises the sum of squared relative
 * errors (predicted / measured - 1)^2, so that short and long messages count
 * alike -- the pages give the model's form, not its constants.  On noisy data
 * a fitted parameter can come out negative (vr_set_cost_model refuses it).
 * Errors: VR_ERR_INVALID_ARGUMENT for n < 2, NULL arrays, a bad R /
 * localRanks, or fewer than two usable samples (or a singular system) for an
 * algorithm. */
vr_result_t vr_fit_cost_model(int n, const int* R, const int* localRanks,
                              const size_t* bytesPerRank, const double* ringUs,
                              const double* treeUs, vr_cost_model_t* out);

/* The message size per rank at which the ring and tree predictions are equal
 * under `model` (NULL: the current model), from the closed form of the two
 * lines; *bytes = -1 when they do not cross at a positive size.  Errors as
 * vr_predict_us. */
vr_result_t vr_crossover_bytes(int R, int localRanks, const vr_cost_model_t* model,
                               double* bytes);

/* Installs `model` as the current model for this process (NULL restores the
 * built-in one), e.g. one fitted to other hardware.  Errors:
 * VR_ERR_INVALID_ARGUMENT for negative or non-finite entries. */
vr_result_t vr_set_cost_model(const vr_cost_model_t* model);

/* ------------------------------------------ run-time specialised trees
 * Tree AllReduce on 16-byte aligned buffers runs kernels compiled at run time
 * (NVRTC, opened with dlopen) for the call's trees: the fold program of each
 * tree ([Course13] "每种 rank 的操作", post-order) becomes straight-line code
 * instead of an interpreted control stream, with the same operations in the
 * same order, so results are unchanged.  Kernels are cached per architecture,
 * element type, op and set of trees; the first call with new trees compiles
 * them (about a second).  Without NVRTC, without the kernel sources beside
 * the library, or with the option VR_JIT=0 (see the top of this header), the
 * built-in interpreting kernels run. */

/* Whether specialised trees are in use, and how many kernel sets were
 * compiled and failed to compile or load so far.  Errors:
 * VR_ERR_INVALID_ARGUMENT for a NULL output. */
vr_result_t vr_jit_status(int* enabled, long long* compiled, long long* failed);

/* Compiles, without loading or touching a device, the specialised kernels of
 * vr_build_dtree(nNodes, localRanks, 2)'s two trees for sm_<smArch>a (e.g.
 * 103) -- register path, staged, staged drawing its tiles (VR_SCHED) -- and
 * returns their total CUBIN size; the compiler log, if any, goes to `log`
 * (logBytes, NUL-terminated, may be NULL / 0).  Errors:
 * VR_ERR_INVALID_ARGUMENT for bad sizes, dtype, op or smArch < 90;
 * VR_ERR_UNSUPPORTED when NVRTC or the kernel sources are not found;
 * VR_ERR_INTERNAL when the compilation fails. */
vr_result_t vr_jit_compile_dtree(int nNodes, int localRanks, vr_dtype_t dtype, vr_op_t op,
                                 int smArch, size_t* cubinBytes, char* log, size_t logBytes);

/* The same for the ring fold of R ranks (register-path and staged kernels):
 * the R ranks' units loaded in rank order, block j's rotation folded from
 * them ([Interview] "手撕代码": block j starts at rank j), one straight-line
 * case per j.  Register-path ring kernels of 16-byte aligned buffers with
 * 3 <= R <= 16 use it (measured 6-12% faster; neutral on the staged kernel,
 * which keeps the loop); the environment variable VR_JIT_RING=0 (read per
 * call) turns it off, VR_JIT_RING=1 also applies it to the staged kernel.
 * Errors as
 * vr_jit_compile_dtree (R outside [1, VR_MAX_RANKS]: invalid). */
vr_result_t vr_jit_compile_ring(int R, vr_dtype_t dtype, vr_op_t op, int smArch,
                                size_t* cubinBytes, char* log, size_t logBytes);

/* ------------------------------------------------------------- status */

/* Synchronises `stream`, then returns and clears the current device's status
 * word: VR_SUCCESS, or the first device-side error any kernel of this library
 * recorded since the last call (VR_ERR_TIMEOUT for a bounded wait that ran
 * out, VR_ERR_INTERNAL for a broken invariant: in the bounds-checked build,
 * an access outside the call's buffers, refused; VR_ERR_INVALID_ARGUMENT for
 * a bad value in device memory, a target of vr_linear_xent), or VR_ERR_CUDA
 * when the
 * synchronisation itself fails.  The word is per device, not per stream. */
vr_result_t vr_stream_status(void* stream);

/* Number of kernels this library has launched in this process (all devices,
 * all threads). */
unsigned long long vr_launch_count(void);

/* Test hook for the device-side failure path.  The next collective call
 * that runs a shared-memory-staged kernel (16-byte aligned AllReduce or
 * ReduceScatter) or the TMA AllGather makes its first CTA skip the loads of
 * its tile number
 * `tile`, so the wait for that tile runs out after the bounded-wait limit
 * (1 s, or VR_WAIT_TIMEOUT_NS nanoseconds from the environment at first
 * use): that call's results are incomplete and vr_stream_status reports
 * VR_ERR_TIMEOUT; the stream and the context stay usable.  -1 cancels a
 * pending request.  Errors: VR_ERR_INVALID_ARGUMENT for tile < -1. */
vr_result_t vr_debug_stall_next(long long tile);

/* Test hook for the tile scheduler of the staged AllReduce kernels (see
 * VR_SCHED): reads (write = 0) or writes (write != 0) the four words of the
 * scheduler slot that calls on `stream` use -- owner (0 when free), next
 * tile, and the CTAs that joined (low 32 bits) and left (high 32 bits) --
 * through a copy on `stream`, which is then synchronised.  A slot whose owner
 * is set to a value no launch has makes the next call's CTAs wait for it
 * (bounded) and report VR_ERR_TIMEOUT; writing four zeros frees it.
 * `words` is host memory of 4 elements.  Errors: VR_ERR_INVALID_ARGUMENT
 * (null words, or a stream being captured), VR_ERR_UNSUPPORTED (no slot
 * left for a new stream), VR_ERR_CUDA. */
vr_result_t vr_debug_sched_slot(void* stream, unsigned long long* words, int write);

/* Sets one of the options listed at the top of this header for the rest of
 * the process (all threads, all devices); value -1 restores the built-in
 * default.  Calls already enqueued are not affected.  Meant for tests and
 * tuning: options choose among kernels that compute the same bits.
 * Errors: VR_ERR_INVALID_ARGUMENT for an unknown name or value < -1. */
vr_result_t vr_set_option(const char* name, long long value);

/* The current value of an option (-1: the call site's built-in default).
 * Errors: VR_ERR_INVALID_ARGUMENT for an unknown name or NULL value. */
vr_result_t vr_get_option(const char* name, long long* value);

/* ------------------------------------------------ bounds-checked build
 * The library's calls return at enqueue, so a kernel's fault would surface
 * later and asynchronously ([Internals] "API 返回只意味着提交边界").  The
 * bounds-checked build of this library (libvr_debug.so, built by
 * double_binary_tree_gb300.build with debug=True; loaded by the Python
 * binding when VR_BOUNDS_CHECKED=1) compiles every global-memory access of
 * every collective's kernel with a check against the buffers of its call (the
 * operators of a training step run the same there as in the normal build;
 * their tensor copies are clipped by the hardware): the send and
 * receive buffers (count elements, or the collective's sizes) and the
 * stepwise ring's FIFO.  An access outside them (a store outside the
 * receive buffers and the FIFO) is skipped, VR_ERR_INTERNAL is recorded in
 * the status word (vr_stream_status) and the first such address in a second
 * device word.  Results and performance of the normal build are unchanged:
 * there the checks compile to nothing. */

/* 1 in the bounds-checked build, 0 in the normal one. */
int vr_debug_bounds_checked(void);

/* The first address the bounds-checked build refused on the current device
 * since the last call (0: none), then cleared.  Errors: VR_ERR_INVALID_ARGUMENT
 * for NULL address, VR_ERR_CUDA when the device cannot be read. */
vr_result_t vr_debug_bounds_fault(unsigned long long* address);

/* Test hook of the bounds-checked build: the next kernel launch records some
 * of its buffers as ending `bytes` earlier than they do (`which`: 1 the
 * send buffers, 2 the receive buffers, 4 the FIFO, or a sum), so the checks
 * refuse its last accesses to them while every access still lies inside
 * real memory: refused loads read zeros (a refused bulk copy into shared
 * memory completes its barrier without copying), refused stores are not
 * made, and vr_stream_status reports VR_ERR_INTERNAL.  No effect in the
 * normal build.  bytes == 0 cancels a pending request.
 * Errors: VR_ERR_INVALID_ARGUMENT for bytes < 0 or which outside 0..7. */
vr_result_t vr_debug_shrink_next(long long bytes, int which);

/* The bounds predicate of the device checks, run on the host (for tests):
 * 1 when [p, p + size) lies inside one of the n extents [lo[i], lo[i] +
 * bytes[i]) -- a writable one (writable[i] != 0) when store != 0 -- else 0;
 * -1 for bad arguments (n < 0, n > 129, NULL arrays with n > 0).  NULL
 * extents never match.  Touches no memory at p. */
int vr_debug_access_ok(const void* const* lo, const unsigned long long* bytes,
                       const int* writable, int n, const void* p, unsigned long long size,
                       int store);

/* Static English text for a result code ("unknown result" for others). */
const char* vr_get_error_string(vr_result_t result);

/* Releases host-side caches (tree programs, device properties).  Optional;
 * the library stays usable afterwards. */
void vr_finalize(void);

#ifdef __cplusplus
}
#endif

#endif /* VR_H */
