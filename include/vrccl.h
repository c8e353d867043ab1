/*
 * vrccl -- ring AllReduce over n virtual ranks resident in one GPU's memory.
 *
 * C ABI of libvrccl.so. Plain C: no CUDA, C++ or torch types appear here;
 * a CUDA stream is passed as an opaque pointer (a cudaStream_t cast to
 * void*, NULL = the legacy default stream), and every buffer is a raw
 * device address on the communicator's device.
 *
 * Sources cited:
 *   [Deep Dive]    "NCCL Source Code Deep Dive: A GPU Journey of One
 *                  AllReduce" (aireadcode.com; English edition, chapters
 *                  1-4; the Japanese edition adds ch.5 tuning and ch.6
 *                  enqueue).
 *   [Architecture] "NCCL architecture: topology, channels, algorithms and
 *                  protocols" (arganzheng.life, part 4 of the series
 *                  "Communication and interconnect: from NCCL to RDMA").
 *
 * What it computes. An AllReduce over n ranks: every rank r contributes
 * sendbufs[r][0..count) and every rank receives, in recvbufs[r][0..count),
 * the elementwise op over all n contributions [Deep Dive §1.3]. The ranks
 * are virtual: n buffers in one GPU's HBM. Each channel owns a contiguous
 * 16-byte-aligned part of the elements and runs the whole algorithm on it
 * independently [Deep Dive §2.2; Architecture §6.3]. On a channel the ring
 * algorithm is a reduce-scatter followed by an all-gather, n-1 steps each,
 * chunked as RingARAlgorithm::getNextSendAddr describes [Deep Dive §2.3;
 * Architecture §9.4, runRing]; rank r hands chunks to rank r+1 (mod n)
 * through staging FIFOs in global memory, synchronised by one of the three
 * wire protocols Simple, LL and LL128 [Architecture §7.2]; with Simple the
 * all-gather writes each finished chunk straight into the next rank's recv
 * buffer instead (runRing's direct primitives; vrcclCommSetDirect). The tree
 * algorithm reduces up and broadcasts down the double binary tree
 * [Architecture §5.4, §9.4; Deep Dive ch.4, ncclGetBtree/ncclGetDtree].
 *
 * Numerics. Eight element types (vrcclDataType_t). bf16, fp16 and fp32 ops
 * are computed in binary32 (no contraction) and rounded (to nearest even)
 * to the element type after every step; fp64 ops are computed in binary64.
 * Integer sum/prod (int8, uint8, int32, int64) wrap modulo 2^bits; max/min
 * compare signed, unsigned for uint8. For the ring, an element of chunk j
 * ends up as
 *   op(...op(op(x[j+1], x[j+2]), x[j+3])..., x[j])        (ranks mod n)
 * where the first operand is the value that arrived from the previous rank
 * and max/min keep the first operand on a tie. avg (not an NCCL op on the
 * pages): the floating types multiply every input once by 1/n before the
 * sum (the binary32 1.0f/n for bf16/fp16/fp32, the binary64 1.0/n for
 * fp64); the integer types divide the wrapped sum by n, truncating toward
 * zero, once per chunk.
 *
 * Ordering and concurrency. Every call is asynchronous on its stream and
 * returns once the work is enqueued [Deep Dive §1.3, "Step 2"]; results are
 * defined after the stream is synchronised. Calls on one communicator
 * share its FIFOs: they must be ordered (one stream, or streams ordered by
 * events); calls that overlap on the GPU are undefined. Different
 * communicators are independent. Calls may be captured in a CUDA graph:
 * the FIFO counters and flags live in device memory and continue from one
 * replay to the next, so a replayed call gives the same results as a
 * direct one, provided the communicator's launches (captured or not) stay
 * ordered. A replay does not run the host's LL flag-wrap accounting (the
 * FIFOs are cleared before a 32-bit LL flag could repeat); that takes
 * about 2^31 LL steps per ring edge, i.e. millions of replayed LL calls.
 *
 * Errors. Synchronous errors return a code and launch nothing. A device-
 * side failure (a wait that timed out, or an abort) is reported later by
 * vrcclCommGetAsyncError; after it the communicator accepts only
 * vrcclCommGetAsyncError, vrcclCommGetErrorInfo and vrcclCommDestroy
 * (as a revoked NCCL communicator fails fast, [Deep Dive (Japanese
 * edition) ch.6, ncclEnqueueCheck step 1]).
 */
#ifndef VRCCL_H_
#define VRCCL_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define VRCCL_VERSION_MAJOR 0
#define VRCCL_VERSION_MINOR 1

/* Largest number of virtual ranks one communicator accepts. */
#define VRCCL_MAX_RANKS 128
/* Largest channel count (NCCL's MAXCHANNELS, [Architecture §5.2]). */
#define VRCCL_MAX_CHANNELS 64
/* FIFO depth per edge and protocol: slots a sender may fill ahead of its
 * receiver (NCCL_STEPS is 8, [Architecture §6.5]; one GPU's HBM hop costs a
 * few microseconds, so twice NCCL's depth keeps ~100 KB in flight per edge). */
#define VRCCL_STEPS 16

typedef struct vrcclComm* vrcclComm_t;
typedef void* vrcclStream_t; /* a cudaStream_t */

/* Result codes, after ncclResult_t [Deep Dive (Japanese edition) ch.5]. */
typedef enum {
  vrcclSuccess = 0,
  vrcclInvalidArgument = 1, /* a bad pointer, size, enum or handle */
  vrcclInvalidUsage = 2,    /* a valid request this communicator or GPU cannot serve */
  vrcclInternalError = 3,
  vrcclCudaError = 4,       /* a CUDA runtime call failed */
  vrcclTimeout = 5,         /* a device-side wait gave up (asynchronous) */
  vrcclAborted = 6,         /* vrcclCommAbort was called (asynchronous) */
  vrcclNumResults = 7
} vrcclResult_t;

/* Element types [Deep Dive §1.3, ncclDataType_t]. Integer sum and prod
 * wrap modulo 2^bits, max and min compare signed (unsigned for uint8), avg
 * is the wrapped sum divided by n, truncating toward zero. bf16 / fp16 /
 * fp32 combine in binary32 and round to the type at every hop; fp64
 * combines in binary64; avg pre-scales each input by 1/n (binary32 for
 * the 2- and 4-byte types, binary64 for fp64). */
typedef enum {
  vrcclInt32 = 0,
  vrcclFloat32 = 1,
  vrcclBfloat16 = 2,
  vrcclFloat16 = 3,
  vrcclInt8 = 4,
  vrcclUint8 = 5,
  vrcclInt64 = 6,
  vrcclFloat64 = 7,
  vrcclNumTypes = 8
} vrcclDataType_t;

typedef enum {
  vrcclSum = 0,
  vrcclProd = 1,
  vrcclMax = 2,
  vrcclMin = 3,
  vrcclAvg = 4,
  vrcclNumOps = 5
} vrcclRedOp_t;

/* Schedules [Architecture §7.1]. vrcclAlgoOneShot is not on the pages: an
 * AllReduce that reads all n inputs of an element at once and writes all n
 * outputs (no FIFO), in the ring's association order for the ring's channel
 * count and chunk. It moves only the essential bytes and serves as the HBM
 * bound the ring is measured against; "auto" never picks it. */
typedef enum {
  vrcclAlgoRing = 0,
  vrcclAlgoTree = 1,
  vrcclAlgoAuto = 2,
  vrcclAlgoOneShot = 3
} vrcclAlgo_t;

/* Wire protocols [Architecture §7.2; Deep Dive §2.4]. */
typedef enum {
  vrcclProtoSimple = 0, /* slot of raw data, then a released tail counter */
  vrcclProtoLL = 1,     /* 16-byte lines: 4 B data, 4 B flag, 4 B data, 4 B flag */
  vrcclProtoLL128 = 2,  /* 128-byte lines: 120 B data, 8 B flag */
  vrcclProtoAuto = 3
} vrcclProto_t;

/*
 * vrcclCommInit -- create a communicator of `nranks` virtual ranks on the
 * current CUDA device, able to run up to `nchannels` channels.
 * Model: ncclCommInitAll, one process driving every rank [Deep Dive §1.2].
 * Allocates, on that device, the FIFOs of every protocol for up to
 * nchannels channels, their control words and status words (about
 * 3 * nranks * nchannels * 1.1 MiB), and zeroes them.
 *   comm      out: the new handle; owned by the caller until
 *             vrcclCommDestroy.
 *   nranks    1..VRCCL_MAX_RANKS.
 *   nchannels 1..VRCCL_MAX_CHANNELS; an upper bound, calls may use fewer.
 * Errors: vrcclInvalidArgument (null comm, out-of-range sizes);
 *         vrcclCudaError (no device, allocation failed; nothing is leaked).
 * Environment, read once here: VRCCL_TIMEOUT_MS (device wait limit,
 * default 2000), VRCCL_DEBUG=INFO (prints each call's decision line),
 * VRCCL_ALGO / VRCCL_PROTO (NCCL_ALGO / NCCL_PROTO's list syntax, see
 * vrcclParseList: what "auto" may choose; an unknown name makes this call
 * return vrcclInvalidArgument), VRCCL_NCHANNELS (channel count "auto" uses),
 * VRCCL_SLICE_BYTES (largest Simple FIFO slot to use, bytes; default and
 * most 32768), VRCCL_SIMPLE_WARPS (most consumer warps per Simple agent, at
 * most 16; default 16 for 2-byte types, 8 for 4-byte ones), VRCCL_PREFETCH (input slices a Simple agent pulls into L2
 * ahead of use, default 0 = off, at most 32), VRCCL_DIRECT (default 1; 0
 * selects the FIFO all-gather, see vrcclCommSetDirect), VRCCL_TUNE_FILE (a measured
 * tuning table, see vrcclCommLoadTuning; without it the table shipped next
 * to the library, tuning/gb300_n<nranks>.txt, is used when present).
 */
vrcclResult_t vrcclCommInit(vrcclComm_t* comm, int nranks, int nchannels);

/*
 * vrcclAllReduce -- AllReduce of `count` elements over the communicator's
 * n virtual ranks, enqueued on `stream` as one kernel launch.
 * Model: ncclAllReduce(sendbuff, recvbuff, count, datatype, op, comm,
 * stream) [Deep Dive §1.3], with the n per-rank pointers of a
 * single-process clique passed together and the algorithm and protocol
 * selectable per call.
 *   sendbufs  host array of n device pointers; sendbufs[r] holds `count`
 *             elements of `dtype`. Read during the call only.
 *   recvbufs  host array of n device pointers; recvbufs[r] receives
 *             `count` elements. recvbufs[r] == sendbufs[r] (in place) is
 *             allowed; any other overlap between the 2n buffers is not.
 *   count     elements per rank. 0 -> success, nothing launched, and the
 *             buffer pointers are not examined (they may be NULL)
 *             [Deep Dive (Japanese edition) ch.6, taskAppend step 4].
 *   dtype, op as above.
 *   algo      ring, tree, auto (the tuning table's choice among ring and
 *             tree), or one-shot (same bits as the ring with the same
 *             channel count and chunk; `proto` is then ignored).
 *   proto     simple, ll, ll128, or auto (the tuning table's choice).
 *   comm      a live communicator.
 *   stream    cudaStream_t on the communicator's device.
 * Every pointer must be 16-byte aligned. With n == 1 the result is a
 * copy of the input (after the avg scale), launched as the same kernel.
 * Errors: vrcclInvalidArgument (null/misaligned/overlapping pointers, bad
 * enum, null comm); vrcclInvalidUsage (communicator already failed, or the
 * forced schedule cannot be made co-resident on this GPU); vrcclCudaError
 * (launch failure).
 */
vrcclResult_t vrcclAllReduce(const void* const* sendbufs, void* const* recvbufs, size_t count,
                             vrcclDataType_t dtype, vrcclRedOp_t op, vrcclAlgo_t algo,
                             vrcclProto_t proto, vrcclComm_t comm, vrcclStream_t stream);

/*
 * vrcclReduceScatter -- the reduce-scatter phase of the ring AllReduce run
 * alone [Deep Dive §2.3: the AllReduce is a reduce-scatter phase and an
 * all-gather phase of n-1 steps each]. Block r of every rank's send buffer
 * is reduced into rank r's recv buffer, one launch on `stream`. The pages
 * give the phase, not a buffer contract; NCCL's ncclReduceScatter contract
 * is followed.
 *   sendbufs  host array of n device pointers; sendbufs[r] holds n blocks
 *             of `recvcount` elements (block q = elements [q*recvcount,
 *             (q+1)*recvcount)). Read during the call only.
 *   recvbufs  host array of n device pointers; recvbufs[r] receives
 *             `recvcount` elements: element e = op over ranks of their
 *             block r, element e, associated in ring order
 *             op(...op(x[r+1], x[r+2])..., x[r]). In place:
 *             recvbufs[r] == sendbufs[r] + r*recvcount elements.
 *   recvcount elements per block; recvcount * element size must be a
 *             multiple of 16 bytes when n > 1, so that every block starts
 *             on a 16-byte boundary. 0 -> success, nothing launched, the
 *             pointers not examined.
 *   dtype, op as for vrcclAllReduce (avg: the same pre-scale / post-op).
 *   proto     simple, ll, ll128, or auto. The schedule is the ring.
 * Channels split each block; a loop takes one chunk of every block. Errors
 * as for vrcclAllReduce, plus vrcclInvalidArgument for a block that is not
 * a multiple of 16 bytes.
 */
vrcclResult_t vrcclReduceScatter(const void* const* sendbufs, void* const* recvbufs, size_t recvcount,
                                 vrcclDataType_t dtype, vrcclRedOp_t op, vrcclProto_t proto,
                                 vrcclComm_t comm, vrcclStream_t stream);

/*
 * vrcclAllGather -- the all-gather phase of the ring AllReduce run alone
 * [Deep Dive §2.3]: rank q's send buffer lands as block q of every rank's
 * recv buffer, bit for bit, one launch on `stream`. NCCL's ncclAllGather
 * contract is followed.
 *   sendbufs  host array of n device pointers; sendbufs[r] holds
 *             `sendcount` elements. Read during the call only.
 *   recvbufs  host array of n device pointers; recvbufs[r] receives n
 *             blocks of `sendcount` elements. In place:
 *             sendbufs[r] == recvbufs[r] + r*sendcount elements.
 *   sendcount elements per block, with the same 16-byte rule as
 *             vrcclReduceScatter. 0 -> success, nothing launched.
 *   dtype     any type; the data moves as 4-byte words (no arithmetic).
 *   proto     simple, ll, ll128, or auto. The schedule is the ring.
 * Errors as for vrcclReduceScatter.
 */
vrcclResult_t vrcclAllGather(const void* const* sendbufs, void* const* recvbufs, size_t sendcount,
                             vrcclDataType_t dtype, vrcclProto_t proto, vrcclComm_t comm,
                             vrcclStream_t stream);

/*
 * vrcclGroupStart / vrcclGroupEnd -- ncclGroupStart / ncclGroupEnd
 * [Architecture §9.2, §9.6; Deep Dive (Japanese edition) ch.5]. Between
 * the two, vrcclAllReduce / vrcclReduceScatter / vrcclAllGather check their
 * arguments (and return any error at once) but only register the call; the
 * outermost vrcclGroupEnd schedules every registered call of every
 * communicator and enqueues it. Groups nest; the depth is per thread.
 * Scheduling, per communicator: AllReduces of one type, op and requested
 * protocol whose algo is ring or auto are sorted by size, largest first,
 * and cut into runs of sizes within 4x of the run's largest
 * (ncclPrepareTasks). A run is scheduled as a whole, by the tuning table at
 * its total size, and enqueued as one launch of the grouped ring kernel
 * (more launches if its pointers exceed the kernel's parameter space);
 * each of its calls gets the channel count a call of its own size would
 * get. Every other call is enqueued alone. The calls of one group are not
 * ordered among themselves: none may touch a buffer another one writes.
 * All of a group's calls on one communicator must use one stream
 * (vrcclInvalidUsage otherwise, at the call). vrcclGroupEnd returns the
 * first error of a launch and drops the calls not yet enqueued; without a
 * matching vrcclGroupStart it returns vrcclInvalidUsage. Like every call
 * here, it only enqueues: synchronise the stream before reading results.
 * vrcclAllReduceNoAlloc is never grouped.
 */
vrcclResult_t vrcclGroupStart(void);
vrcclResult_t vrcclGroupEnd(void);

/*
 * vrcclCommGetGroupSchedule -- what ran for call `index` (0-based, in call
 * order) of the communicator's most recent group: algorithm, protocol,
 * channel count, chunk (elements; together with the channel count it
 * fixes the association order of every float result), and the launch
 * (0-based, in enqueue order within the group) that carried it. Calls that
 * shared a launch report the same launch.
 * Errors: vrcclInvalidArgument (bad handle, index out of range);
 * vrcclInvalidUsage (nothing ran for that call: count 0).
 */
vrcclResult_t vrcclCommGetGroupSchedule(vrcclComm_t comm, int index, int* algo, int* proto, int* nchannels,
                                        size_t* chunkElems, int* launch);

/*
 * vrcclParseList -- the list syntax of VRCCL_ALGO / VRCCL_PROTO, which is
 * NCCL_ALGO / NCCL_PROTO's (parseList, [Architecture §8.5]): elements are
 * comma separated; a leading '^' excludes the listed names instead; a
 * "function:" prefix restricts a list to one collective; ';' separates
 * lists, the first of which may have no prefix (it applies to every
 * collective). Names are case-insensitive and are NCCL's: functions
 * Broadcast, Reduce, AllGather, ReduceScatter, AllReduce; algorithms Tree,
 * Ring, CollNetDirect, CollNetChain, NVLS, NVLSTree, PAT; protocols LL,
 * LL128, Simple. Of those this library has Ring and Tree (AllReduce; the
 * others are ring-only) and all three protocols; "auto" chooses among the
 * allowed ones, and a call left with none returns vrcclInvalidUsage.
 *   spec   the string (NULL or empty: everything allowed).
 *   kind   0 = algorithms, 1 = protocols.
 *   masks  out: 5 masks, one per function in the order above; bit i is the
 *          i-th name of the kind in the order above.
 * Errors: vrcclInvalidArgument for an unknown name (then vrcclCommInit
 * refuses the same string in the environment).
 */
vrcclResult_t vrcclParseList(const char* spec, int kind, unsigned* masks);

/*
 * vrcclModelPredict -- the pages' analytic model of an AllReduce's time,
 * T = latency * numPipeOps(ring) + bytes / (1000 * algorithm bandwidth) us
 * (ncclTopoTuneModel / ncclTopoGetAlgoTime, [Architecture §8.1-§8.3]),
 * with the constants the pages print. It serves to set the measured tuning
 * table beside the pages' model; the library never schedules by it.
 *   graph      ranks, nodes, channels, per-channel link bandwidth (GB/s)
 *              inside a node and across nodes, extra latency per inter-node
 *              step (us), intra-node hardware (0 NVLink, 1 PCI), GPU
 *              architecture (0 Volta, 1 Ampere, 2 Hopper, 3 Blackwell).
 *   algo       ring or tree; proto: simple, ll or ll128.
 *   bytes      message size; numPipeOps: operations aggregated with it (>= 1).
 *   latUs, algBwGBs, timeUs  out (each may be NULL).
 * Errors: vrcclInvalidArgument for an inconsistent graph or a bad enum.
 */
typedef struct {
  int nranks;
  int nnodes;
  int nchannels;
  float bwIntra;
  float bwInter;
  float latencyInter;
  int hwIntra;
  int arch;
} vrcclModelGraph_t;
vrcclResult_t vrcclModelPredict(const vrcclModelGraph_t* graph, vrcclAlgo_t algo, vrcclProto_t proto, size_t bytes,
                                int numPipeOps, float* latUs, float* algBwGBs, float* timeUs);

/*
 * vrcclCommSetDirect -- 1 (the default): the communicator's later ring /
 * Simple AllReduces and AllGathers run the all-gather through the ranks'
 * recv buffers instead of the FIFOs (the directRecvCopyDirectSend primitives of runRing, which
 * read and write a peer's user buffer where the ranks can address each
 * other, [Architecture §9.4, §10]): the step that finishes chunk r writes
 * it to rank r's recv buffer and straight into rank r+1's, each later step
 * forwards it from the rank's own recv buffer into the next rank's, and a
 * counter per ring edge, released after the writes, tells the next rank it
 * is there. The reduce-scatter still moves through the FIFOs. Results are
 * bit-identical to the FIFO form, which moves (6n-4) S bytes through the
 * SMs against the direct form's (5n-4) S. A standalone AllGather moves
 * each block the same way: written into the next rank's recv buffer, then
 * forwarded from there; grouped AllReduces do the same task by task. 0 (or
 * VRCCL_DIRECT=0 at vrcclCommInit) selects the FIFO all-gather. LL, LL128,
 * the tree and ReduceScatter always use the FIFOs.
 * Errors: vrcclInvalidArgument (bad handle, enable not 0 or 1).
 */
vrcclResult_t vrcclCommSetDirect(vrcclComm_t comm, int enable);

/*
 * vrcclCommSetSchedule -- pin the channel count and chunk size used by
 * later calls (0 = choose automatically, the default).
 *   nchannels  0, or 1..the communicator's nchannels.
 *   chunkBytes 0, or the ring chunk size K*E in bytes: a multiple of 16
 *              and at most VRCCL_STEPS/2 FIFO slots of the protocol in use
 *              (ALLREDUCE_CHUNKSTEPS = NCCL_STEPS/2, [Deep Dive (Japanese
 *              edition) ch.6]); a larger value is clamped at call time.
 * Errors: vrcclInvalidArgument.
 */
vrcclResult_t vrcclCommSetSchedule(vrcclComm_t comm, int nchannels, size_t chunkBytes);

/*
 * vrcclCommGetLastSchedule -- the schedule the last successful
 * vrcclAllReduce on this communicator used: algo, proto, channel count
 * and ring chunk size in elements (K). Any output pointer may be NULL.
 * With this a checker can replay the exact association order.
 * Errors: vrcclInvalidArgument (null comm); vrcclInvalidUsage (no call yet).
 */
vrcclResult_t vrcclCommGetLastSchedule(vrcclComm_t comm, int* algo, int* proto, int* nchannels,
                                       size_t* chunkElems);

/*
 * vrcclCommGetAsyncError -- the communicator's device-side status:
 * vrcclSuccess, vrcclTimeout or vrcclAborted
 * [Deep Dive §1.4, ncclCommGetAsyncError]. Does not wait for running
 * work; reads the status word through an internal stream.
 * Errors: vrcclInvalidArgument; vrcclCudaError.
 */
vrcclResult_t vrcclCommGetAsyncError(vrcclComm_t comm, vrcclResult_t* asyncErr);

/*
 * vrcclCommGetErrorInfo -- where the first device-side failure happened:
 * the virtual rank, channel and FIFO step of the wait that gave up (all -1
 * / 0 when there was none). Any output pointer may be NULL.
 */
vrcclResult_t vrcclCommGetErrorInfo(vrcclComm_t comm, int* rank, int* channel, uint64_t* step);

/*
 * vrcclCommSetTimeout -- device wait limit in milliseconds for later
 * launches (1..3600000). Every device spin-wait gives up after this long,
 * records vrcclTimeout and makes every other agent of the launch return.
 */
vrcclResult_t vrcclCommSetTimeout(vrcclComm_t comm, uint64_t timeoutMs);

/*
 * vrcclCommAbort -- raise the communicator's abort word, which every
 * device wait polls; running and later launches return early and the
 * communicator reports vrcclAborted [Deep Dive §1.4; Architecture §9.5,
 * abortFlag]. The communicator must still be destroyed.
 */
vrcclResult_t vrcclCommAbort(vrcclComm_t comm);

/*
 * vrcclCommDestroy -- wait for the communicator's work to finish
 * (device-synchronising), free everything it allocated, and invalidate
 * the handle. NULL is accepted and ignored.
 */
vrcclResult_t vrcclCommDestroy(vrcclComm_t comm);

/* vrcclCommCount -- the number of virtual ranks [Deep Dive §1.2]. */
vrcclResult_t vrcclCommCount(vrcclComm_t comm, int* nranks);

/* vrcclGetErrorString -- a static, human-readable name of a result code. */
const char* vrcclGetErrorString(vrcclResult_t result);

/*
 * vrcclCommInjectFault -- testing aid: in every later launch, agent
 * (rank, channel) of the given algorithm returns without doing its work
 * once it reaches FIFO step `afterSteps` of the launch, so its peers' waits
 * run out (a flag that nothing sets). rank = -1 clears the fault. Nothing
 * faults or traps: the launch ends when the waits give up.
 */
vrcclResult_t vrcclCommInjectFault(vrcclComm_t comm, int rank, int channel, int afterSteps);

/*
 * vrcclCommGetLaunchShape -- the launch geometry of the last successful
 * vrcclAllReduce: CTAs (one per agent), threads per CTA and elements per
 * FIFO slot. Any output pointer may be NULL.
 * Errors: vrcclInvalidArgument; vrcclInvalidUsage (no call yet).
 */
vrcclResult_t vrcclCommGetLaunchShape(vrcclComm_t comm, int* blocks, int* threads, int* sliceElems);

/*
 * vrcclCommLoadTuning -- replace the communicator's tuning table with the
 * entries of a measured table file that match its rank count. NCCL fills
 * latency/bandwidth tables from constants and takes the smallest predicted
 * time T = lat + bytes/bw [Architecture §8.2]; this table holds measured
 * times instead, and algo/proto/channels "auto" take its minimum at the
 * nearest measured power-of-two size. File format, one entry per line:
 *   nranks algo proto channels log2bytes sliceBytes microseconds [elementBytes]
 * ('#' starts a comment; algo/proto use the enum values above). A line with
 * elementBytes (1, 2, 4 or 8) applies to calls whose element type has that
 * size; a line without it applies to every element type. A call takes the
 * rows of its own element size if the table has any, else the rows without
 * one, else those of the nearest element size (the larger on a tie).
 *   loaded  out (may be NULL): entries kept.
 * Errors: vrcclInvalidArgument (null comm/path, unreadable file).
 */
vrcclResult_t vrcclCommLoadTuning(vrcclComm_t comm, const char* path, int* loaded);

/*
 * vrcclShardRange -- the part of one virtual-rank problem that GPU `shard`
 * of `nshards` computes, when the problem's element range is split across
 * GPUs [Architecture §6.3: channels own independent contiguous ranges and
 * never synchronise, so the channel partition of Deep Dive §2.2 applies one
 * level up]. Parts are contiguous, in shard order, of alignUp(ceil(count /
 * nshards), 16 bytes) elements; trailing parts may be short or empty. Each
 * GPU holds the n virtual ranks' slices [offset, offset + length) of their
 * buffers and runs vrcclAllReduce on them with a communicator of its own
 * (no data moves between GPUs: the outputs are disjoint). Host only.
 *   count    elements per virtual rank of the whole problem.
 *   offset, length  out: the shard's first element and element count.
 * Errors: vrcclInvalidArgument (bad dtype, nshards < 1, shard outside
 * [0, nshards), null outputs).
 */
vrcclResult_t vrcclShardRange(size_t count, vrcclDataType_t dtype, int nshards, int shard, size_t* offset,
                              size_t* length);

/*
 * vrcclAllReduceNoAlloc -- the ring / Simple AllReduce of vrcclAllReduce,
 * for callers that cannot allocate device memory when they need it (code
 * running under a memory-pool manager that owns all of the device's
 * memory, or a latency-critical path that cannot take cudaMalloc's implicit
 * device synchronisation) and keep no communicator. The pages have no
 * counterpart: NCCL always reduces through a communicator's buffers.
 *   sendbufs, recvbufs, count, dtype, op, stream: as for vrcclAllReduce
 *             (caller-owned, 16-byte aligned device buffers; in place
 *             allowed).
 *   nranks    1..32 virtual ranks (the count of sendbufs / recvbufs).
 * Schedule: ring, Simple, min(4, 32 / nranks) channels, chunk 256 KiB
 * (= vrcclCommSetSchedule(comm, that many channels, 262144) on the
 * communicator path, with identical results).
 * Memory: allocates nothing. Its scratch (FIFO slots, counters, status;
 * about 16 MiB) is one static device array that every GPU loading the
 * library holds until the process exits. The first call on a device looks
 * up that array's address, prepares the kernels and reads VRCCL_TIMEOUT_MS;
 * make that first call before any stream capture (a set-up that fails is
 * not kept: the next call tries again). Every call then zeroes the
 * counters and status words on `stream` and launches one kernel; calls
 * share the array, so calls that overlap on the GPU (other streams, other
 * host threads) race and give undefined results -- order them.
 * Errors: vrcclInvalidArgument (null/misaligned pointers, bad enum,
 * nranks < 1, buffers that overlap other than in place); vrcclInvalidUsage
 * (nranks > 32: the scratch is too small -- use a communicator);
 * vrcclCudaError / vrcclInternalError (set-up or launch failed).
 * Device-side failures are not reported (there is no communicator to
 * ask): a wait still gives up after VRCCL_TIMEOUT_MS (default 2 s) and
 * the kernel returns, but the call has already returned vrcclSuccess and
 * the recv buffers are then undefined.
 */
vrcclResult_t vrcclAllReduceNoAlloc(const void* const* sendbufs, void* const* recvbufs, size_t count, int nranks,
                                    vrcclDataType_t dtype, vrcclRedOp_t op, vrcclStream_t stream);

/* ------------------------------------------------------------------------
 * Operators of a replica: what a data-parallel rank computes between two
 * AllReduces of its gradients -- layer norm, RMS norm, dropout, the linear
 * layer, a distillation loss and the log probabilities of given tokens, each
 * forward and backward. They need no communicator: a call
 * runs on the current CUDA device, is asynchronous on `stream` like every
 * call here, allocates nothing (what scratch it needs the caller passes as
 * `workspace`) and may be captured in a CUDA graph.
 *
 * Matrices are row-major with a row stride in elements (ldx, ...), which may
 * exceed the row's length; only the elements of the rows are written, and
 * beside them nothing is read but what shares a 16-byte block with a row
 * between the matrix's first element and its last (it is ignored). Pointers must be aligned to their element's size; rows that all
 * start on 16-byte boundaries are faster. The operators take vrcclFloat32,
 * vrcclBfloat16 and vrcclFloat16 (the linear layer only the latter two).
 * Sums and statistics are held in binary32 and each result is rounded once
 * (to nearest even); there are no atomic sums, so the same call gives the
 * same bits.
 *
 * Errors of all of them: vrcclInvalidArgument (a null or misaligned pointer,
 * a row stride below the row's length, an enum or a size out of range, a
 * workspace that is too small, an output that overlaps an input or another
 * output other than as the call allows); vrcclCudaError (launch failure).
 * Matrices of one row stride in bytes may lie side by side in a wider buffer
 * (column slices), and vectors between a matrix's rows; of two strides the
 * whole address ranges may not meet.
 */

/*
 * vrcclLayerNormForward -- y = (x - mean) * rstd * gamma + beta over the
 * columns of each row, rstd = 1 / sqrt(mean((x - mean)^2) + eps).
 *   x, y         [rows, cols] of dtype; y may be x (same stride).
 *   gamma, beta  [cols] of paramType, or NULL (1 and 0).
 *   mean, rstd   out, [rows] binary32: what the backward pass takes; either
 *                may be NULL.
 *   rows, cols   0 of either -> success, nothing launched.
 *   eps          >= 0.
 */
vrcclResult_t vrcclLayerNormForward(const void* x, size_t ldx, const void* gamma, const void* beta, void* y,
                                    size_t ldy, float* mean, float* rstd, size_t rows, size_t cols,
                                    vrcclDataType_t dtype, vrcclDataType_t paramType, float eps,
                                    vrcclStream_t stream);

/* vrcclLayerNormWorkspace -- bytes of workspace the backward pass of this
 * size needs (the partial sums of the weights' gradients). */
vrcclResult_t vrcclLayerNormWorkspace(size_t rows, size_t cols, size_t* bytes);

/*
 * vrcclLayerNormBackward -- with xh = (x - mean) * rstd and g = dy * gamma:
 *   dx = rstd * (g - mean(g) - xh * mean(g * xh))      per row
 *   dgamma = sum over rows of dy * xh,  dbeta = sum over rows of dy
 *   dy, x, dx      [rows, cols] of dtype; dx may be dy or x (same stride).
 *   gamma          [cols] of paramType, or NULL (1).
 *   mean, rstd     [rows], as the forward pass wrote them.
 *   dgamma, dbeta  out, [cols] of paramType; either may be NULL. With
 *                  rows == 0 they are set to zero.
 *   workspace      16-byte aligned, vrcclLayerNormWorkspace bytes; NULL where
 *                  neither gradient is asked for.
 */
vrcclResult_t vrcclLayerNormBackward(const void* dy, size_t lddy, const void* x, size_t ldx, const void* gamma,
                                     const float* mean, const float* rstd, void* dx, size_t lddx, void* dgamma,
                                     void* dbeta, size_t rows, size_t cols, vrcclDataType_t dtype,
                                     vrcclDataType_t paramType, void* workspace, size_t workspaceBytes,
                                     vrcclStream_t stream);

/* Activations of the linear layer: gelu is z * Phi(z) with the normal
 * distribution Phi, gelu-tanh its approximation
 * z/2 * (1 + tanh(sqrt(2/pi) * (z + 0.044715 z^3))), silu z / (1 + exp(-z)). */
typedef enum {
  vrcclActNone = 0,
  vrcclActRelu = 1,
  vrcclActGelu = 2,
  vrcclActGeluTanh = 3,
  vrcclActSilu = 4,
  vrcclNumActs = 5
} vrcclActivation_t;

/* vrcclLinearWorkspace -- bytes of workspace a call of this size may need
 * (backward: 0 or 1), whatever its strides. A forward call whose x and w
 * have all their rows on 16-byte boundaries needs none. */
vrcclResult_t vrcclLinearWorkspace(int backward, size_t rows, size_t outs, size_t ins, vrcclDataType_t dtype,
                                   vrcclActivation_t act, size_t* bytes);

/*
 * vrcclLinearForward -- z = x w^T + bias, y = act(z) + residual.
 *   x         [rows, ins];  w [outs, ins];  y [rows, outs].
 *   bias      [outs], or NULL.
 *   residual  [rows, outs], or NULL; y may be residual (same stride).
 *   z         out, [rows, outs]: what the backward pass of an activation
 *             takes, or NULL.
 *   dtype     vrcclBfloat16 or vrcclFloat16, of every operand. Products and
 *             sums are binary32. vrcclFloat32 -> vrcclInvalidUsage: the
 *             tensor cores would round its operands to 10 fraction bits.
 *   workspace 256-byte aligned wherever one is passed; may be NULL where none
 *             is needed.
 */
vrcclResult_t vrcclLinearForward(const void* x, size_t ldx, const void* w, size_t ldw, const void* bias,
                                 const void* residual, size_t ldr, void* y, size_t ldy, void* z, size_t ldz,
                                 size_t rows, size_t outs, size_t ins, vrcclDataType_t dtype, vrcclActivation_t act,
                                 void* workspace, size_t workspaceBytes, vrcclStream_t stream);

/*
 * vrcclLinearBackward -- with dz = dy * act'(z):
 *   dx = dz w,  dw = dz^T x,  dbias = sum over rows of dz
 * (the residual's gradient is dy itself).
 *   dy, z     [rows, outs]; z as the forward pass wrote it, not read for
 *             vrcclActNone.
 *   x, w      [rows, ins], [outs, ins].
 *   dx, dw, dbias  out, [rows, ins], [outs, ins], [outs]; each may be NULL.
 *             A sum over no rows is zero.
 * With an activation dz is rounded to dtype before the two products, which
 * take their operands in it; dbias sums the unrounded values.
 */
vrcclResult_t vrcclLinearBackward(const void* dy, size_t lddy, const void* z, size_t ldz, const void* x, size_t ldx,
                                  const void* w, size_t ldw, void* dx, size_t lddx, void* dw, size_t lddw, void* dbias,
                                  size_t rows, size_t outs, size_t ins, vrcclDataType_t dtype, vrcclActivation_t act,
                                  void* workspace, size_t workspaceBytes, vrcclStream_t stream);

/* vrcclReplicaGetAsyncError -- vrcclSuccess, or vrcclTimeout after an
 * operator's kernel on the current device gave up a wait (its outputs are
 * then undefined). Waits for the device's work on every stream (so not while
 * one is being captured). The status is the device's, of the whole process,
 * and is not cleared: once vrcclTimeout, every later query reports it. */
vrcclResult_t vrcclReplicaGetAsyncError(vrcclResult_t* asyncErr);

/* Most teacher entries a row of the distillation loss may have. */
#define VRCCL_DISTILL_MAX_K 1024

/*
 * vrcclDistillForward -- the loss of a student against a teacher known by
 * its top logits: with temperature T, p = softmax(teacher / T) over a row's
 * kept entries and q = softmax(logits / T) over the vocabulary,
 *   loss = T^2 * sum over entries of p * (log p - log q[index]).
 * An entry is kept if its index lies in [0, vocab) and its logit is not
 * -inf; entries that share an index add up. A NaN is kept, so that it shows:
 * the row's loss and the gradients of its entries are then NaN. A row without
 * kept entries has loss 0 and gradient 0 (a padding position), whatever its
 * logits hold. Masked student logits may be -inf or the type's lowest value.
 *   logits   [rows, vocab] of dtype.
 *   teacher  [rows, k] of teacherType;  index [rows, k] of indexType
 *            (vrcclInt32 or vrcclInt64), k <= VRCCL_DISTILL_MAX_K.
 *   loss     out, [rows] binary32.
 *   stats    out, [rows, 2] binary32, 8-byte aligned, or NULL: the row's
 *            largest logit and the logarithm of the sum of
 *            exp((logits - largest) / T); 0, 0 for a row without entries.
 *   temperature  1e-18 to 1e18.
 */
vrcclResult_t vrcclDistillForward(const void* logits, size_t ldl, const void* teacher, size_t ldt, const void* index,
                                  size_t ldi, float* loss, float* stats, size_t rows, size_t vocab, size_t k,
                                  vrcclDataType_t dtype, vrcclDataType_t teacherType, vrcclDataType_t indexType,
                                  float temperature, vrcclStream_t stream);

/*
 * vrcclDistillBackward -- the gradient of those losses,
 *   dlogits[v] = dloss * T * (q[v] - sum of p over the entries with index v),
 * zero in rows without kept entries.
 *   stats    as the forward pass wrote them.
 *   dloss    binary32, row r's at dloss[r * dlossStride] (stride 0: one
 *            value for all rows).
 *   dlogits  out, [rows, vocab] of dtype; may be logits (same stride).
 */
vrcclResult_t vrcclDistillBackward(const void* logits, size_t ldl, const void* teacher, size_t ldt, const void* index,
                                   size_t ldi, const float* stats, const float* dloss, size_t dlossStride,
                                   void* dlogits, size_t ldd, size_t rows, size_t vocab, size_t k,
                                   vrcclDataType_t dtype, vrcclDataType_t teacherType, vrcclDataType_t indexType,
                                   float temperature, vrcclStream_t stream);

/*
 * vrcclDropoutForward -- y = residual + (kept ? x * scale : 0), the kept
 * elements drawn by a counter-based generator, so that nothing of the mask is
 * stored: the backward pass (and a recomputed forward pass) draws it again.
 *   x, y      [rows, cols] of dtype; y may be x (same stride).
 *   residual  [rows, cols], or NULL (0); y may be residual (same stride).
 *   p         0 to 1, the probability of being dropped, taken as the nearest
 *             multiple of 2^-16: drop = round(65536 p); scale = 65536 /
 *             (65536 - drop). A dropped element adds nothing, whatever x holds.
 *   seed      DEVICE address of one 64-bit word, read when the kernel runs (so
 *             that a captured graph draws another mask once the word changes).
 *   offset    which of the masks of one seed: calls that are to differ (layers,
 *             steps) take offsets of their own.
 *   firstRow  number of row 0. The mask of a row depends on its number, so that
 *             a batch that is cut over calls or ranks has the mask of the whole.
 * Element (r, c) is kept if its 16 bits are not below drop: with n = (firstRow
 * + r) ceil(cols / 8) + c / 8 and Philox4x32-10 (Salmon et al., 2011) under
 * the key `seed` for the counter (n, offset), low words first, the lower (c
 * even) or upper half of the output's word c % 8 / 2. Strides, type and
 * alignment do not enter.
 * Errors: vrcclInvalidArgument (also p outside [0, 1] or NaN, firstRow >= 2^40).
 */
vrcclResult_t vrcclDropoutForward(const void* x, size_t ldx, const void* residual, size_t ldr, void* y, size_t ldy,
                                  size_t rows, size_t cols, vrcclDataType_t dtype, float p, const uint64_t* seed,
                                  uint64_t offset, size_t firstRow, vrcclStream_t stream);

/*
 * vrcclDropoutBackward -- dx = kept ? dy * scale : 0 under the mask that the
 * forward call with the same p, seed, offset, firstRow and cols drew (the
 * residual's gradient is dy itself).
 *   dy, dx  [rows, cols] of dtype; dx may be dy (same stride).
 */
vrcclResult_t vrcclDropoutBackward(const void* dy, size_t lddy, void* dx, size_t lddx, size_t rows, size_t cols,
                                   vrcclDataType_t dtype, float p, const uint64_t* seed, uint64_t offset, size_t firstRow,
                                   vrcclStream_t stream);

/* 8-bit codes of the RMS norm: int8 (-127 to 127), or e4m3 (4 exponent and 3
 * fraction bits, largest 448). */
typedef enum {
  vrcclQuantInt8 = 0,
  vrcclQuantE4M3 = 1,
  vrcclNumQuants = 2
} vrcclQuant_t;

/*
 * vrcclRmsNormForward -- s = x + residual, rounded to dtype, and
 * y = s * rstd * gamma, rstd = 1 / sqrt(mean(s^2) + eps) over the columns of
 * each row.
 *   x, residual  [rows, cols] of dtype; residual may be NULL (s = x).
 *   gamma        [cols] of paramType, or NULL (1).
 *   sum          out, [rows, cols] of dtype: s, what the backward pass and the
 *                next addition take; or NULL.
 *   y            out, [rows, cols] of dtype, or NULL where codes are asked for.
 *                sum and y may each be x or residual (same stride), not both
 *                the same one.
 *   codes        out, [rows, cols] bytes, or NULL: y in 8 bits, code = y /
 *                scale (to binary32's precision) rounded to the nearest (even)
 *                int8 or e4m3.
 *   scales       out, binary32 [rows, ceil(cols / group)], what a code is
 *                multiplied by: the largest |y| of the group (unrounded) over
 *                the largest code, at least 2^-126. Not finite where a y of the
 *                group is not.
 *   quant, group read with codes alone: the codes' type, and how many columns
 *                share a scale: 32, 64, 128, or 0 for the whole row.
 *   rstd         out, [rows] binary32, what the backward pass takes; or NULL.
 *   rows, cols   0 of either -> success, nothing launched.
 *   eps          >= 0. A row's squares are summed in binary32: where the sum
 *                passes its range (|s| beyond some 1e19) rstd is 0; where it is
 *                0 and eps too, infinite.
 * vrcclAllGather carries codes as vrcclInt8 or vrcclUint8.
 */
vrcclResult_t vrcclRmsNormForward(const void* x, size_t ldx, const void* residual, size_t ldr, const void* gamma,
                                  void* sum, size_t lds, void* y, size_t ldy, void* codes, size_t ldc, float* scales,
                                  size_t ldsc, float* rstd, size_t rows, size_t cols, vrcclDataType_t dtype,
                                  vrcclDataType_t paramType, vrcclQuant_t quant, size_t group, float eps,
                                  vrcclStream_t stream);

/* vrcclRmsNormWorkspace -- bytes of workspace the backward pass of this size
 * needs (the partial sums of the weight's gradient); 0 for 0 rows or columns. */
vrcclResult_t vrcclRmsNormWorkspace(size_t rows, size_t cols, size_t* bytes);

/*
 * vrcclRmsNormBackward -- with xh = s * rstd and g = dy * gamma:
 *   dx = dsum + rstd * (g - xh * mean(g * xh))      per row
 *   dgamma = sum over rows of dy * xh
 * dx is the gradient of x and of residual alike. Codes pass the gradient on as
 * if they were y.
 *   dy, s, dx  [rows, cols] of dtype; s as the forward pass wrote (or took) it;
 *              dx may be dy, dsum or s (same stride).
 *   dsum       [rows, cols]: the gradient that reaches s other than through
 *              the norm, or NULL (0).
 *   gamma      [cols] of paramType, or NULL (1).
 *   rstd       [rows], as the forward pass wrote it.
 *   dgamma     out, [cols] of paramType, or NULL. With rows == 0 it is set to
 *              zero.
 *   workspace  16-byte aligned, vrcclRmsNormWorkspace bytes; NULL where dgamma
 *              is not asked for.
 */
vrcclResult_t vrcclRmsNormBackward(const void* dy, size_t lddy, const void* dsum, size_t ldds, const void* s, size_t lds,
                                   const void* gamma, const float* rstd, void* dx, size_t lddx, void* dgamma, size_t rows,
                                   size_t cols, vrcclDataType_t dtype, vrcclDataType_t paramType, void* workspace,
                                   size_t workspaceBytes, vrcclStream_t stream);

/* Most alternatives a row of vrcclLogProbForward lists. */
#define VRCCL_LOGPROB_MAX_K 32

/*
 * vrcclLogProbForward -- with q = softmax(logits / T) over the vocabulary:
 *   logprob = log q[token],  entropy = - sum of q * log q,
 * and the k likeliest entries.
 *   logits    [rows, vocab] of dtype.
 *   token     [rows] of tokenType (vrcclInt32 or vrcclInt64), or NULL: none
 *             are given (logprob is then NULL too). A row whose token lies
 *             outside [0, vocab) is a padding position: its logits count for
 *             nothing, its logprob, entropy and stats are 0.
 *   logprob, entropy  out, [rows] binary32; either may be NULL.
 *   stats     out, [rows, 2] binary32, 8-byte aligned, or NULL: the row's
 *             largest logit and the logarithm of the sum of
 *             exp((logits - largest) / T), what the backward pass takes.
 *   top, topIndex  out, [rows, k] binary32 and 32-bit integers: the log
 *             probabilities and indices of the k largest logits, the largest
 *             first, equal ones by the lowest index (zeros of either sign are
 *             equal; a NaN counts as the largest). Where there are fewer (k >
 *             vocab, a padding position): -inf and -1. NULL with k == 0.
 *   k         0 to VRCCL_LOGPROB_MAX_K.
 *   temperature  1e-18 to 1e18.
 * Masked logits may be -inf or the type's lowest value. A row of nothing but
 * -inf has no distribution: logprob -inf, entropy 0, stats (-inf, 0). A NaN or
 * +inf among the logits makes the row's values NaN.
 */
vrcclResult_t vrcclLogProbForward(const void* logits, size_t ldl, const void* token, float* logprob, float* entropy,
                                  float* stats, float* top, size_t ldt, int32_t* topIndex, size_t ldi, size_t rows,
                                  size_t vocab, size_t k, vrcclDataType_t dtype, vrcclDataType_t tokenType,
                                  float temperature, vrcclStream_t stream);

/*
 * vrcclLogProbBackward -- the gradient of logprob and entropy,
 *   dlogits[v] = (dlogprob * ((v == token) - q[v]) - dentropy * q[v] * (log q[v] + entropy)) / T,
 * zero at padding positions and in rows of nothing but -inf. (The
 * alternatives are for reading; no gradient flows through them.)
 *   stats, entropy  as the forward pass wrote them; entropy is read with
 *             dentropy alone.
 *   dlogprob  binary32, row r's at dlogprob[r * dlogprobStride] (stride 0: one
 *             value for all rows), or NULL (0); needs token.
 *   dentropy  likewise; one of the two is given.
 *   token     as forward (NULL if none were given).
 *   dlogits   out, [rows, vocab] of dtype; may be logits (same stride).
 */
vrcclResult_t vrcclLogProbBackward(const void* logits, size_t ldl, const void* token, const float* stats,
                                   const float* entropy, const float* dlogprob, size_t dlogprobStride,
                                   const float* dentropy, size_t dentropyStride, void* dlogits, size_t ldd, size_t rows,
                                   size_t vocab, vrcclDataType_t dtype, vrcclDataType_t tokenType, float temperature,
                                   vrcclStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* VRCCL_H_ */
