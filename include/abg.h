/*
 * abg.h -- C ABI of the GB300 (sm_103a) affine 4-bit group-quantized
 * matrix-vector product and its two activation producers.
 *
 * The operation comes from three Bend pull-request pages by one author:
 *   [q4mv-metal]  "Array.q4mv on Metal: one kernel thread per row for products
 *                 of 4M weights or more, bit-identical" (bendlang/bend #1435)
 *   [q4go]        "Array.q4go/Array.q4wait queue Metal Q4 products in one
 *                 command buffer and wait once on a flag" (#1437)
 *   [fused-token] "Metal: queued rmsq, swq, gdn and atq kernels and a 4-row
 *                 q4mv, so a decode token is one command buffer with one wait"
 *                 (#1440)
 *
 * Weight format ([fused-token] Why and Change; [q4go] Verification): MLX-style
 * 4-bit affine weights, w = scale*q + bias with q in 0..15, in groups of 64
 * columns.  q is packed 8 nibbles per u32: column 8k+j of a row is bits
 * 4j..4j+3 of word k (low nibble first).  scale and bias are f32, one per row
 * and 64-column group.  The product reads the activation x together with its
 * 64-value group sums xsum, so that
 *
 *     y[r] = sum_g ( scale[r][g] * sum_j q[r][64g+j] * x[64g+j]
 *                    + bias[r][g] * xsum[g] ).
 *
 * Modes.  ABG_TREE reproduces a fixed summation order bit for bit ([fused-token]
 * Change, bend_q4mv bullet: "sums in a fixed tree order").  Every sum is a
 * balanced pairwise tree in index order: at each level elements (2i, 2i+1)
 * are added and an odd last element is carried up unchanged.  Products are
 * rounded once (RN binary32), the affine term is RN(RN(scale*d) + RN(bias*xsum))
 * without fused multiply-add, and each row's group terms are summed by the
 * same tree.  ABG_FAST may reorder and contract; its outputs stay within
 * 1e-5 * max(|y|, sum_g |scale*d| + |bias*xsum|) of the tree result.
 *
 * Conventions shared by every call:
 *   - Pointers are DEVICE pointers owned by the caller (the library allocates
 *     nothing per call).  Packed weights and every vector read in pairs
 *     (x, wt, a, and the xn / o outputs) must be 16-byte aligned; group sums,
 *     scale, bias and y 4-byte aligned (else ABG_EALIGN).  scale and bias
 *     rows are streamed with bulk copies when both are 16-byte aligned and
 *     cols is a multiple of 256, and read with ordinary loads otherwise.
 *   - Calls are asynchronous: they enqueue on `stream` (a cudaStream_t, NULL =
 *     the legacy default stream) and return.  The caller synchronizes.
 *   - Lifetime ([q4go] Change, last paragraph; Limits): every buffer a call
 *     reads or writes must stay allocated and unmodified by others until the
 *     stream work has completed.  Freeing w early was seen to corrupt row 0.
 *   - An output may not overlap any input of the same call (else ABG_EALIAS):
 *     concurrent products must not read one another's y ([q4go] Change).
 *   - Lengths that are not whole 64-value groups are rejected (ABG_ESHAPE).
 *     The pages' GPU kernels silently left such outputs untouched
 *     ([fused-token] reviewer reply); here it is an error.
 *   - A device-side wait that exceeds its time limit (0.5 s) stops the
 *     kernel and sets a bit in the library's device status word; read it with
 *     abg_device_status().  No call hangs the GPU.
 */
#ifndef ABG_H
#define ABG_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ABG_OK = 0,
    ABG_EINVAL = 1,   /* null pointer, bad mode, bad enum, bad count */
    ABG_EALIGN = 2,   /* a pointer is not aligned as the call requires */
    ABG_ESHAPE = 3,   /* size not a positive multiple of 64, row range out of bounds, cols too large */
    ABG_EALIAS = 4,   /* an output overlaps an input (or, in a graph, a same-stage read) */
    ABG_ECUDA = 5,    /* a CUDA runtime call failed; see abg_last_cuda_error() */
    ABG_ETIMEOUT = 6  /* a device-side wait ran out of time (reported by abg_device_status) */
} abg_status;

typedef enum { ABG_TREE = 0, ABG_FAST = 1 } abg_mode;

/* Storage type of scale and bias ([fused-token] Why: the MLX 4-bit formats).
 * 16-bit values are widened to f32 exactly before use (bf16: the upper half
 * of an f32; f16: IEEE binary16), so the arithmetic is the same as for f32
 * storage of the widened values. */
typedef enum { ABG_SB_F32 = 0, ABG_SB_BF16 = 1, ABG_SB_F16 = 2 } abg_sb_type;

/* Largest `cols` a product accepts: the activation row is staged once per
 * thread block in shared memory. */
#define ABG_MAX_COLS 16384

/*
 * q4mv: rows row0 .. row0+n-1 of the packed rows x cols matrix times x.
 * ([q4go] Change: Array.q4go(w, x, y, r, n, cols, rows) -- reading: r is the
 *  first row, n the number of rows computed, rows the matrix height that
 *  locates each row's words, scale and bias.)
 *
 *   w      u32 [rows][cols/8]   packed nibbles (see the header comment)
 *   scale  f32 [rows][cols/64]
 *   bias   f32 [rows][cols/64]
 *   x      f32 [cols]
 *   xsum   f32 [cols/64]        xsum[g] = tree sum of x[64g .. 64g+63]
 *   y      f32 [n]              y[i] = row row0+i
 *   cols   positive multiple of 64, at most ABG_MAX_COLS
 *   0 <= row0, 0 <= n, row0 + n <= rows.  n == 0 enqueues nothing.
 *   mode   ABG_TREE or ABG_FAST
 *   rows_per_warp  1, 2, 4 or 8 rows share one staging of each 1024-column
 *          slice of x in a warp's registers ([fused-token] Change: a SIMD
 *          group does 4 rows and reads each group's activations once); 0 picks
 *          the default (8).  It never changes the result.
 */
abg_status abg_q4mv(const uint32_t *w, const float *scale, const float *bias,
                    const float *x, const float *xsum, float *y,
                    int64_t rows, int64_t cols, int64_t row0, int64_t n,
                    int mode, int rows_per_warp, void *stream);

/*
 * q4mv_ex: the same product for the other MLX 4-bit formats ([fused-token]
 * Why): groups of `group` columns (32, 64 or 128) and scale/bias stored as
 * `sb_type` (abg_sb_type).
 *
 *     y[r] = sum_g ( scale[r][g] * sum_j q[r][group*g+j] * x[group*g+j]
 *                    + bias[r][g] * xsum[g] ),   g < cols/group,
 *
 * with the same tree order and rounding as abg_q4mv (which is this call with
 * group 64 and ABG_SB_F32).
 *   scale, bias  [rows][cols/group] of f32, or of 16-bit bf16 / f16 patterns;
 *                aligned to their element size (4 or 2 bytes)
 *   xsum   f32 [cols/group]   xsum[g] = tree sum of x[group*g .. group*g+group-1]
 *   cols   a positive multiple of 64 and of group, at most ABG_MAX_COLS
 * scale and bias rows are streamed with bulk copies when both pointers are
 * 16-byte aligned and a row of them is a multiple of 16 bytes.  Other
 * arguments and errors as abg_q4mv; a bad group or sb_type is ABG_EINVAL.
 */
abg_status abg_q4mv_ex(const uint32_t *w, const void *scale, const void *bias, int sb_type, int group,
                       const float *x, const float *xsum, float *y,
                       int64_t rows, int64_t cols, int64_t row0, int64_t n,
                       int mode, int rows_per_warp, void *stream);

/*
 * q4mm: the product for a batch of T decode tokens that share the weights
 * (the 4-row q4mv of [fused-token] Change reads each activation group once for
 * several rows; here each weight is read once for several tokens):
 *
 *     y[t*n + i] = q4mv row row0+i of x[t*cols .. t*cols+cols-1],  t < T,
 *
 * each token's result bit-identical to abg_q4mv on that token alone (ABG_TREE).
 *   x     f32 [T][cols], 16-byte aligned (rows follow each other)
 *   xsum  f32 [T][cols/64]   xsum[t][g] = tree sum of token t's group g
 *   y     f32 [T][n]
 *   T     1..8.  Each group of four tokens (rows of 2048 columns with
 *         bulk-copied scale and bias) or pair of tokens is one launch that
 *         reads the weights once for all of them; an odd last token runs as
 *         a single-token product.
 *         The first launch waits for the stream's earlier work; the later
 *         ones may start while it runs (programmatic dependent launch, off
 *         with ABG_PDL=0), since they read the same inputs and write other
 *         rows of y.
 * Groups of 64 columns with f32 scale and bias; other arguments and errors as
 * abg_q4mv.
 */
abg_status abg_q4mm(const uint32_t *w, const float *scale, const float *bias,
                    const float *x, const float *xsum, float *y,
                    int64_t rows, int64_t cols, int64_t row0, int64_t n, int64_t T,
                    int mode, int rows_per_warp, void *stream);

/*
 * gsum: s[g] = tree sum of v[64g .. 64g+63], g < n/64.  The group sums a
 * product reads for its bias term ([fused-token] Change, Array.rmsq bullet:
 * "the 64-value group sums that Array.q4mv reads").  n a positive multiple of 64.
 */
abg_status abg_gsum(const float *v, float *s, int64_t n, int mode, void *stream);
/* gsum_ex: s[g] = tree sum of v[group*g .. group*g+group-1], group 32, 64 or
 * 128; n a positive multiple of 64 and of group. */
abg_status abg_gsum_ex(const float *v, float *s, int64_t n, int group, int mode, void *stream);

/*
 * rmsq: RMS norm with weights plus the group sums of its output
 * ([fused-token] Change, Array.rmsq bullet).
 *   ss      = tree over groups of (tree over the group of x[i]*x[i])
 *   r       = 1 / sqrt(ss / n + eps)
 *   xn[i]   = (x[i] * r) * wt[i]
 *   xsum[g] = tree sum of xn over group g
 * x, wt, xn f32 [n]; xsum f32 [n/64]; n a positive multiple of 64, at most
 * 2^20.  Runs in one thread block.
 */
abg_status abg_rmsq(const float *x, const float *wt, float eps, float *xn, float *xsum,
                    int64_t n, int mode, void *stream);
/* rmsq_ex: the same with xsum over groups of `group` values (32, 64 or 128;
 * xsum f32 [n/group]; n also a multiple of group).  The norm factor does not
 * depend on the group size: the two-level tree of squares is the pairwise tree
 * over all n values. */
abg_status abg_rmsq_ex(const float *x, const float *wt, float eps, float *xn, float *xsum,
                       int64_t n, int group, int mode, void *stream);

/*
 * swq: SwiGLU plus the group sums of its output ([fused-token] Change,
 * Array.swq(a, o, n) bullet).  a = [gate (n) | up (n)].
 *   o[i]    = silu(a[i]) * a[n+i],  silu(g) = g / (1 + EXP(-g))
 *   osum[g] = tree sum of o over group g
 * In ABG_TREE mode EXP is the library's own binary32 exponential (Cody-Waite
 * reduction with a two-part ln 2, degree-7 Taylor polynomial with RN(1/i!)
 * coefficients, exact scaling by 2^k), so the result is bit-exact across
 * devices; a vendor exp moves the last bits ([fused-token] Change, last
 * paragraph).  a f32 [2n]; o f32 [n]; osum f32 [n/64]; n a positive multiple
 * of 64.
 */
abg_status abg_swq(const float *a, float *o, float *osum, int64_t n, int mode, void *stream);
/* swq_ex: the same with osum over groups of `group` values (32, 64 or 128;
 * osum f32 [n/group]; n also a multiple of group). */
abg_status abg_swq_ex(const float *a, float *o, float *osum, int64_t n, int group, int mode, void *stream);

/*
 * gdn: one token of a gated DeltaNet mixer ([fused-token] Change, Array.gdn
 * bullet: conv window and activation, q/k L2 norms, decay and beta, the
 * delta-rule rows, the gated norm and group sums; one threadgroup per value
 * head, every phase local to its head).  The page gives no formulas; this is
 * the published gated DeltaNet recurrence with one key head per value head,
 * every step one binary32 operation rounded to nearest, every sum the
 * library's pairwise tree, EXP as in swq and LOG the library's own logarithm
 * (reduction to [sqrt(1/2), sqrt(2)) times 2^e, 2 atanh(s) by its series to
 * s^9, e*ln2 in two parts):
 *   SIGMOID(u) = 1/(1 + EXP(-u)), SILU(u) = u/(1 + EXP(-u)),
 *   SOFTPLUS(u) = u if u > 20, else LOG(1 + EXP(u))
 *   channel c of x = [q | k | v]: window w = [state[c][0..K-2], x[c]],
 *     a_c = SILU(tree_t conv[c][t]*w[t]), state[c] <- w[1..K-1]
 *   head h: qh = q * (1/sqrt(tree q*q + eps)) * RN(1/sqrt(D)),
 *     kh = k * (1/sqrt(tree k*k + eps)),
 *     alpha = EXP(-(EXP(A_log[h]) * SOFTPLUS(a[h] + dt_bias[h]))),
 *     beta = SIGMOID(b[h]),
 *     S <- alpha*S;  d_j = beta*(v_j - tree_i S[i][j]*kh_i);
 *     S[i][j] <- S[i][j] + kh_i*d_j;  o_j = tree_i S[i][j]*qh_i,
 *     y_j = ((o_j * 1/sqrt(tree(o*o)/D + eps_n)) * nw_j) * SILU(z[h*D+j])
 *   ysum = 64-value group sums of y.
 *   x        f32 [3*H*D] (q, then k, then v; head h's block at h*D)
 *   conv     f32 [3*H*D][K]         state  f32 [3*H*D][K-1], updated in place
 *   a, b, A_log, dt_bias f32 [H]    z      f32 [H*D]      nw  f32 [D]
 *   S        f32 [H][D][D] (key i, value j), updated in place; 16-byte aligned
 *   y        f32 [H*D]              ysum   f32 [H*D/64]
 *   D = 64, 128 or 256; 2 <= K <= 8; H >= 1, H*D <= 2^20.
 * Both modes compute the same bits.  One launch, started early by
 * programmatic dependent launch unless ABG_PDL=0 (it reads every input after
 * the launch before it has finished).  Errors: null pointer or mode
 * ABG_EINVAL; shape ABG_ESHAPE; a pointer not 4-byte aligned, or S not
 * 16-byte aligned, ABG_EALIGN; an
 * output (state, S, y, ysum) overlapping an input or another output
 * ABG_EALIAS.  Asynchronous on `stream`.
 */
abg_status abg_gdn(const float *x, const float *conv, float *state, const float *a, const float *b, const float *z,
                   const float *A_log, const float *dt_bias, const float *nw, float *S, float *y, float *ysum,
                   int64_t H, int64_t D, int64_t K, float eps, float eps_n, int mode, void *stream);

/*
 * atq: one token of gated attention over key and value caches ([fused-token]
 * Change, Array.atq bullet: q/k RMS norm and rotation, the new k/v into the
 * caches, scores, softmax, weighted values, sigmoid gate and group sums; one
 * threadgroup per query head, the first head of each KV group writing the
 * cache row while the others use the new k/v).  The page gives no formulas;
 * this is grouped-query attention at position pos (query head h reads
 * key/value head h / (Hq/Hkv)) with the library's steps (one RN binary32 op
 * each, pairwise trees, EXP and SIGMOID as in gdn):
 *   RMS(u) = 1/sqrt(tree(u*u)/D + eps);  qn = (q_h*RMS(q_h))*qn_w,
 *     kn = (k_g*RMS(k_g))*kn_w
 *   rotation of column pairs (i, i + D/2) by this position's cos_i, sin_i:
 *     r_i = u_i*cos_i - u_{i+D/2}*sin_i, r_{i+D/2} = u_{i+D/2}*cos_i + u_i*sin_i
 *   Kc[g][pos] = rot(kn), Vc[g][pos] = v_g
 *   s_t = tree_j(rot(qn)_j*Kc[g][t][j]) * RN(1/sqrt D), t = 0..pos
 *   p_t = EXP(s_t - max s) / tree_t EXP(s_t - max s)
 *   y_j = tree_t(p_t*Vc[g][t][j]) * SIGMOID(gate[h*D+j]);  ysum = 64-value
 *   group sums of y
 *   q, gate  f32 [Hq*D]    k, v  f32 [Hkv*D]    qn_w, kn_w  f32 [D]
 *   cos, sin f32 [D/2]     Kc, Vc f32 [Hkv][P][D], rows < pos filled; row pos
 *                          written (by the call)
 *   y        f32 [Hq*D]    ysum  f32 [Hq*D/64]
 *   D = 64, 128 or 256; Hq a multiple of Hkv; 0 <= pos < P; pos + 1 <= 8192;
 *   Hq*D <= 2^20.
 * Both modes compute the same bits.  The positions run in chunks of 64 (four
 * launches, started early by programmatic dependent launch unless
 * ABG_PDL=0): the first reads the key cache rows below pos before it waits
 * for the launch before it on the stream, which therefore must not write
 * them.  The chunks' partial results live in a device buffer the library
 * allocates on a device's first call and grows when a call needs more (the
 * growth synchronizes the device, so a call recorded into a stream capture
 * must not need more than an earlier call outside it: ABG_ECUDA otherwise);
 * calls that can overlap on the GPU (on different streams or host threads)
 * share it and must be ordered by the caller.  A stage graph's atq nodes
 * have buffers of their own.  Errors: null pointer
 * or mode ABG_EINVAL; shape ABG_ESHAPE; a pointer not 4-byte aligned, or Kc
 * or Vc not 16-byte aligned, ABG_EALIGN; an output (Kc, Vc, y, ysum)
 * overlapping an input or another output ABG_EALIAS.  Asynchronous on
 * `stream`.
 */
abg_status abg_atq(const float *q, const float *gate, const float *k, const float *v, const float *qn_w,
                   const float *kn_w, const float *cos, const float *sin, float *Kc, float *Vc, float *y, float *ysum,
                   int64_t Hq, int64_t Hkv, int64_t D, int64_t P, int64_t pos, float eps, int mode, void *stream);

/* ---------------------------------------------------------------------------
 * Stage graph: one decode token's dependent stages recorded into one CUDA
 * graph, replayed with one launch and synchronized once by the caller
 * ([fused-token] Why and Verification: one command buffer, one wait per
 * token; [q4go] Change: products queued together run concurrently, and a
 * dependent stage needs the previous one finished).
 *
 * Nodes carry a stage index.  Nodes with the same index form one stage and
 * may run concurrently; every node of stage s+1 runs after every node of
 * stage s has finished.  Products of one stage that read the same x (for
 * example q/k/v, or gate/up) are run as grouped launches of up to 256
 * products each (abg_stage_graph_launches counts them).  Consecutive
 * launches overlap through programmatic dependent launch: a product fetches
 * its weights before the previous stage has finished and waits only before
 * it reads its activation.  Weights, and the norm weights of an RMS-norm
 * prologue, must therefore not be written by any node of the graph (checked:
 * ABG_EALIAS).
 *
 * Node kinds and the fields each reads (unused fields are ignored):
 *   ABG_NODE_Q4MV  w, scale, bias, rows, cols, row0, n, y, prologue, and
 *                  prologue ABG_PRO_NONE: x [cols], xsum [cols/64]
 *                  prologue ABG_PRO_GSUM: x [cols]; xsum computed in-kernel
 *                  prologue ABG_PRO_RMSQ: x [cols] (un-normalized), wt [cols],
 *                                         eps; the product reads rmsq(x, wt)
 *                  prologue ABG_PRO_SWQ:  x [2*cols] = [gate | up]; the
 *                                         product reads swq(x)
 *                  A prologue recomputes the producer inside each thread
 *                  block with the same trees, so the product's result is
 *                  bit-identical to running the producer node first.
 *   ABG_NODE_RMSQ  x, wt, eps, len -> out (xn), out_sum (xsum)
 *   ABG_NODE_SWQ   x (2*len), len -> out (o), out_sum (osum)
 *   ABG_NODE_GSUM  x, len -> out_sum
 *   ABG_NODE_GDN   args (abg_gdn_args): as abg_gdn; reads and writes state
 *                  and S in place
 *   ABG_NODE_ATQ   args (abg_atq_args): as abg_atq; writes row pos of Kc, Vc
 *                  (the graph owns the buffer of the chunk results of each
 *                  ATQ node, so replays of different graphs do not share it);
 *                  no other node may write its Kc or Vc (ABG_EALIAS)
 *   ABG_NODE_COPY  x, len -> out: copies len floats (a memory copy, no
 *                  arithmetic), so that a replay can take its inputs from
 *                  host memory and return its results there: each of x and
 *                  out is device memory or page-locked host memory (pinned or
 *                  registered); pageable host memory, len <= 0, a pointer not
 *                  4-byte aligned or overlapping ranges give ABG_EINVAL,
 *                  ABG_ESHAPE, ABG_EALIGN and ABG_EALIAS.  The kernel launch
 *                  that follows a copy does not start early.
 * Every kind also reads `group` (0 means 64): the group size of the product's
 * scale, bias and xsum (Q4MV, including the group sums its prologue
 * computes) or of out_sum (RMSQ, SWQ, GSUM); Q4MV reads `sb_type` (an
 * abg_sb_type; scale and bias then point at that type).  Sizes given above
 * as cols/64 or len/64 are cols/group and len/group.
 * ------------------------------------------------------------------------- */
typedef enum {
    ABG_NODE_Q4MV = 0,
    ABG_NODE_RMSQ = 1,
    ABG_NODE_SWQ = 2,
    ABG_NODE_GSUM = 3,
    ABG_NODE_GDN = 4, /* args -> abg_gdn_args */
    ABG_NODE_ATQ = 5, /* args -> abg_atq_args */
    ABG_NODE_COPY = 6 /* x -> out, len floats */
} abg_node_kind;

/* The arguments of abg_gdn and abg_atq, for their stage-graph nodes (the
 * struct is read when the graph is created; the pointers must stay valid for
 * the graph's lifetime, like every node's). */
typedef struct abg_gdn_args {
    const float *x, *conv;
    float *state;
    const float *a, *b, *z, *A_log, *dt_bias, *nw;
    float *S, *y, *ysum;
    int64_t H, D, K;
    float eps, eps_n;
} abg_gdn_args;

typedef struct abg_atq_args {
    const float *q, *gate, *k, *v, *qn_w, *kn_w, *cos, *sin;
    float *Kc, *Vc, *y, *ysum;
    int64_t Hq, Hkv, D, P, pos;
    float eps;
} abg_atq_args;
typedef enum { ABG_PRO_NONE = 0, ABG_PRO_GSUM = 1, ABG_PRO_RMSQ = 2, ABG_PRO_SWQ = 3 } abg_prologue;

typedef struct abg_node {
    int32_t kind;      /* abg_node_kind */
    int32_t stage;     /* stage index; any order, grouped by value */
    const uint32_t *w; /* Q4MV */
    const void *scale; /* f32, or 16-bit patterns (sb_type) */
    const void *bias;
    int64_t rows, cols, row0, n;
    float *y;
    int32_t prologue;  /* abg_prologue, Q4MV only */
    float eps;         /* RMSQ node and ABG_PRO_RMSQ */
    const float *x;    /* activation / producer input (see above) */
    const float *xsum; /* Q4MV with ABG_PRO_NONE */
    const float *wt;   /* RMSQ node and ABG_PRO_RMSQ */
    float *out;        /* RMSQ, SWQ, COPY */
    float *out_sum;    /* RMSQ, SWQ, GSUM */
    int64_t len;       /* RMSQ, SWQ, GSUM vector length n; COPY floats */
    int32_t group;     /* group size 32, 64 or 128; 0 = 64 */
    int32_t sb_type;   /* Q4MV: abg_sb_type of scale and bias */
    const void *args;  /* GDN: abg_gdn_args; ATQ: abg_atq_args */
} abg_node;

/* Validates every node (same rules as the single calls), checks that no node
 * reads an output of its own stage, records the launches on a private stream
 * and instantiates the graph.  *graph_out receives an opaque handle.  The
 * graph owns its executable graph and, for SwiGLU pairs (see
 * abg_stage_graph_swiglu_pairs), one device buffer of n floats per pair. */
abg_status abg_stage_graph_create(const abg_node *nodes, int64_t count, int mode, int rows_per_warp,
                                  void **graph_out);
/* With the environment variable ABG_PDL=0 at creation, launches are recorded
 * without programmatic dependent launch (each waits for the previous one to
 * finish before starting); results are identical. */
/* Enqueues one replay of the whole graph on `stream`; the caller syncs once.
 * With the environment variable ABG_TRACE=1 each launch also synchronizes and
 * prints the launch count, GPU milliseconds and wall milliseconds to stderr. */
abg_status abg_stage_graph_launch(void *graph, void *stream);
/* Number of kernel launches one replay performs (after sibling grouping; an
 * ATQ node performs four, a COPY node none). */
abg_status abg_stage_graph_launches(void *graph, int64_t *launches);
/* SwiGLU pairs: when a Q4MV node with the ABG_PRO_SWQ prologue reads a =
 * [gate | up] (2n values) written by the only two products of the launch
 * right before it (gate y = a[0, n), up y = a[n, 2n), one activation, n rows
 * each, groups of 64 with f32 scale and bias, 2048, 4096 or 6144 columns), the
 * gate/up launch also writes silu(gate) * up once per element into a device
 * buffer of n floats that the graph allocates at creation and frees in
 * abg_stage_graph_destroy, and the reading product takes its group sums from
 * that buffer instead of recomputing the SwiGLU in every thread block.  Every
 * node's outputs keep their bits.  *pairs receives how many were formed. */
abg_status abg_stage_graph_swiglu_pairs(void *graph, int64_t *pairs);
abg_status abg_stage_graph_destroy(void *graph);

/* Reads (and, if clear != 0, resets) the device status word on the current
 * device: bit 0 = a device-side wait timed out; bits 4.. name the wait that
 * gave up (16: a stage's release, 32: a stage's arrival, 64: the partial sums
 * of a tile, 128: a final drain of copies, 256: a wait of the 16-bit
 * abg_tree_attn kernel).  Synchronizes the device.
 * Returns ABG_ETIMEOUT when bit 0 was set, else ABG_OK. */
abg_status abg_device_status(uint32_t *bits, int clear);

/* Failure-detection self-test (no counterpart on the pages, whose queued
 * kernels had no bounded waits): enqueues one small product whose producer
 * warp withholds its only tile, so the computing warps' bounded waits run out
 * after the 0.5 s limit.  The kernel then sets bits 0 and 32 of the device
 * status word and exits with no copy in flight; the GPU context stays usable.
 * Reads no caller memory.  Expect abg_device_status to return ABG_ETIMEOUT
 * (and clear it there) after syncing the stream. */
abg_status abg_selftest_wait_timeout(void *stream);

/* Tuning of the product kernel, process-wide; 0 keeps the default.  Applies
 * to calls and graphs created afterwards.
 *   smem_kb          shared-memory budget per thread block (default 110, so
 *                    two blocks fit on an SM and a dependent launch can start
 *                    while its predecessor still runs)
 *   consumer_warps   warps that compute, 1..16 (default: chosen from cols, at
 *                    most 8); above 8 selects one block per SM (with 8 rows
 *                    per warp item)
 *   blocks_per_sm    thread blocks per SM in the grid, at most what fits
 *                    (default: 2)
 *   stage_kb         target size of one pipeline stage of streamed rows
 *                    (default 40)
 * It never changes results. */
abg_status abg_set_q4mv_tuning(int smem_kb, int consumer_warps, int blocks_per_sm, int stage_kb);

/*
 * swiglu_mlp_static: the MLP block y = down( silu(gate x) * (up x) ) with
 * no device allocation and no buffer from the caller for the intermediate
 * vectors.  The pages have no counterpart of this call: it exists for callers
 * that cannot allocate device memory themselves, such as code whose device
 * memory all belongs to another allocator (a framework's caching allocator,
 * or a server that reserves its memory up front), or code on a latency path
 * where cudaMalloc/cudaFree would synchronize the device.
 *   wg, sg, bg  gate product: u32 [n][cols/8], f32 [n][cols/64] x2
 *   wu, su, bu  up product:   the same shapes
 *   wd, sd, bd  down product: u32 [rows][n/8], f32 [rows][n/64] x2
 *   x     f32 [cols], xsum f32 [cols/64] (x's group sums)
 *   y     f32 [rows]  y[i] = row i of the down product of o[j] =
 *                     silu(gate_y[j]) * up_y[j], silu(g) = g / (1 + EXP(-g))
 *   n     rows of gate and up, columns of down: a positive multiple of 64, at
 *         most 16384 (else ABG_ESHAPE)
 * Groups of 64 columns with f32 scale and bias; every result, tree order and
 * error rule as the separate calls (abg_q4mv twice, abg_swq, abg_q4mv), whose
 * results it equals bit for bit in ABG_TREE mode.
 * The intermediate vectors (gate_y, up_y and o, 3n floats) live in one
 * static device array of 3 * 16384 floats inside the library, which every
 * device that loads the library holds until the process exits.  The first
 * call on a device looks up that array's device address (with the device
 * current), so make the first call on each device before any stream capture
 * begins.  Every call uses the same array: calls that can overlap on the GPU
 * (on different streams, or different host threads) race on it and must be
 * ordered by the caller.  Nothing in the array needs clearing: each call
 * writes every element it reads.  Asynchronous like the other calls.
 */
abg_status abg_swiglu_mlp_static(const uint32_t *wg, const float *sg, const float *bg,
                                 const uint32_t *wu, const float *su, const float *bu,
                                 const uint32_t *wd, const float *sd, const float *bd,
                                 const float *x, const float *xsum, float *y,
                                 int64_t n, int64_t cols, int64_t rows, int mode, void *stream);

/* ---------------------------------------------------------------------------
 * Draft verification: several guessed tokens of each of B requests checked in
 * one step, over a paged key/value cache.  The calls of a step, in order:
 *
 *   abg_page_plan    pages and cache slots of the tokens that enter the cache
 *   abg_tree_plan    ancestor masks and positions of the drafts
 *   abg_kv_put       q/k norm and rotation, k/v rows into the cache's layout
 *   abg_tree_attn    attention of the drafts over the cache and one another
 *   abg_tree_accept  the drafts that the logits agree with
 *
 * A request's drafts stay outside the cache, in rows of draft buffers, until
 * they are accepted: a rejected draft costs no page and nothing is moved.  One
 * draft a request is ordinary decoding; a prompt is tokens that enter the
 * cache at once.
 *
 * Shared by these calls:
 *   cu     i32 [B+1]  request b owns rows cu[b] .. cu[b+1]-1 of the N draft
 *          rows (its span), draft i of it is row cu[b]+i; cu[0] = 0,
 *          nondecreasing, cu[B] <= N.  Rows from cu[B] on are padding.
 *   cache  [pages][Hkv][page][D] of f32, bf16 or f16 (an abg_sb_type), page >=
 *          1 tokens a page; slot s is row s % page of page s / page.  A draft
 *          buffer [Hkv][rows][D] is a cache of one page of `rows` tokens, and
 *          the caches of abg_atq are one page of P tokens.
 *   table  i32 [B][width]  page of tokens page*j .. page*j+page-1 of request b
 * Lengths, spans, tables and slots are read on the GPU; what they name out of
 * range is not touched (each call says what it does instead).  These calls
 * have no mode: whole numbers are exact, kv_put's f32 results are those of
 * abg_atq's steps bit for bit, tree_attn's are within the bounds given there
 * and the same on every run.  None of them uses an atomic on global memory.
 *   The launches may start while an earlier kernel of the stream drains
 * (programmatic dependent launch, unless ABG_PDL=0), and read nothing before
 * that kernel's writes are visible; in a stream capture the first launch of
 * each call starts after everything before it.
 * ------------------------------------------------------------------------- */

/* Largest span of a request, and largest number of mask words of a draft
 * (64 drafts a word). */
#define ABG_MAX_SPAN 256
/* Largest B of abg_page_plan (its scan is held in shared memory). */
#define ABG_MAX_REQUESTS 8192

/*
 * page_plan: request b, which has lens[b] tokens in the cache and held[b]
 * pages in its table row, gets the pages and slots for add[b] more tokens, or
 * gives its pages back (add[b] < 0).
 *   Free pages are entries head .. tail-1 (taken modulo ring_len) of `ring`,
 *   ends = {head, tail}.  need = ceil((lens + add) / page), extra = max(0,
 *   need - held); requests take their extra pages from the head in request
 *   order.  A request is granted if extra is 0 or the extras up to and
 *   including its own fit in tail - head; it is refused if they do not, or if
 *   add exceeds its span, need or held exceeds width, lens or held is
 *   negative, or lens + add exceeds 2^31 - 1.  Pages given back go to the
 *   tail in request order (none of them is granted in the same call); a
 *   request whose held is out of range, or whose pages and those given back
 *   before them do not fit in the ring beside the free ones (so none, where
 *   ring_len is at least the number of pages that there are), gives nothing
 *   back and counts as refused.
 *   table  in place: entries held .. need-1 of granted requests
 *   ring   in place: entries from tail on, for pages given back
 *   slots  i64 [N]  slot of token lens+i for i < add of granted requests, else -1
 *   pos    i32 [N]  lens + i there, else 0
 *   lens_out, held_out i32 [B], ends_out i64 [2]: the values for the next call
 *          (refused: unchanged; given back: 0)
 *   info   i32 [2]  pages taken, requests refused
 * Integers only.  The call can be repeated: it reads nothing that it writes.
 * 1 <= B <= ABG_MAX_REQUESTS, 0 <= N < 2^31, page, width, ring_len in 1 .. 2^31-1.
 */
abg_status abg_page_plan(const int32_t *lens, const int32_t *add, const int32_t *cu, const int32_t *held,
                         const int64_t *ends, int32_t *ring, int32_t *table, int64_t *slots, int32_t *pos,
                         int32_t *lens_out, int32_t *held_out, int64_t *ends_out, int32_t *info, int64_t B, int64_t N,
                         int64_t page, int64_t width, int64_t ring_len, void *stream);

/*
 * tree_plan: each draft's ancestors and position from its parent.
 *   parent i32 [N]  index of the parent among the request's drafts; -1 (or an
 *          index that is no other draft of the request) for a root; below -1
 *          for padding.  Any order; a cycle makes its members one another's
 *          ancestors.
 *   mask   u64 [N][words]  bit j: draft j of the request is the draft itself
 *          or an ancestor of it (0 for padding)
 *   pos    i32 [N]  lens[b] + the number of ancestors (0 for padding)
 * 1 <= words <= 4.  Drafts from 64*words on in a span are padding, as are rows
 * from cu[B] on.
 */
abg_status abg_tree_plan(const int32_t *parent, const int32_t *lens, const int32_t *cu, uint64_t *mask, int32_t *pos,
                         int64_t B, int64_t N, int64_t words, void *stream);

/*
 * kv_put: key and value rows of N tokens into a cache, with abg_atq's RMS norm
 * and rotation of q and k (each optional), rounded once to the cache's type.
 *   k, v   source row i, head h at k + i*k_row + h*k_head (in elements), of
 *          src_type (f32, or the cache's type)
 *   rows   i32 [N] or null: token n reads source row rows[n] (null: n).  A
 *          token whose row is outside 0 .. src_rows-1 is skipped.
 *   slots  i64 [N] or null: token n goes to slot slots[n] (null: n).  A slot
 *          outside 0 .. pages*page-1 is not written.
 *   q, qo  q as k (q_row, q_head, Hq heads, src_type); qo [N][Hq][D] of the
 *          cache's type; both null for none
 *   qn_w, kn_w  f32 [D] or null: x <- (x * 1/sqrt(tree(x*x)/D + eps)) * w
 *   cos, sin    f32 [cos_rows][D/2] or both null: rotation of the column
 *          pairs (i, i + D/2) of q and k by row pos[n] (the rows are NaN where
 *          pos[n] is outside 0 .. cos_rows-1)
 *   pos    i32 [N], with cos and sin only
 * D = 64, 128 or 256.  Slots name distinct rows: what two tokens of one slot
 * leave in it is not specified (each value is one or the other's, not all of
 * one token).  Rows, row strides and head strides are multiples of 16 bytes.
 */
typedef struct abg_kv_put_args {
    const void *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;
    const int32_t *rows;
    const int64_t *slots;
    const float *qn_w, *kn_w, *cos, *sin;
    const int32_t *pos;
    void *qo, *Kc, *Vc;
    int64_t N, src_rows, Hq, Hkv, D, page, pages, cos_rows;
    float eps;
    int32_t src_type, type;
} abg_kv_put_args;
abg_status abg_kv_put(const abg_kv_put_args *a, void *stream);

/*
 * tree_attn: attention of every draft over its request's cached tokens and
 * over the drafts of its request that its mask names (query head h reads
 * key/value head h / (Hq/Hkv)):
 *   s_t = q.K_t / sqrt(D)  for the lens[b] cached tokens,
 *   s_j = q.Kd_j / sqrt(D) for the drafts j whose bit is set,
 *   y   = sum_t p_t V_t / sum_t p_t,  p = exp(s - max s),
 * then, with a gate, y * 1/(1 + exp(-gate)).  A draft that sees no token (no
 * cached token and an empty mask, or scores of -infinity only) gives 0.  What
 * a draft does not see does not reach it, not a NaN either.
 *   q      [N][Hq][D]   Kc, Vc  the cache   Kd, Vd [Hkv][drafts][D], drafts >=
 *          N: draft row n's key and value; all of `type`
 *   lens   i32 [B]  (at most width*page is used; a page outside 0 .. pages-1
 *          reads as zeros)
 *   mask   u64 [N][words], 1 <= words <= 4; drafts of a span from 64*words on
 *          are neither attended to nor computed
 *   gate   f32 [N][Hq][D] or null
 *   y      [N][Hq][D] of y_type: `type` or f32
 *   ysum   f32 [N][Hq*D/64] or null, with y_type f32 only: y's 64-value group
 *          sums, for abg_q4mv's xsum
 *   max_span  the largest span (1 .. 64*words): a hint that picks the tiling
 *   ws     abg_tree_attn_workspace() bytes of device memory, for this call's
 *          stream until it is done; its contents need not be kept or cleared
 * Rows outside the spans are not written.  If a wait of the 16-bit kernel
 * gives up (bit 256 of abg_device_status), y and ysum hold no result; nothing
 * else is touched.
 * Sums, softmax statistics and the work split's partial results are f32.  f32
 * operands are multiplied in f32.  16-bit operands are multiplied exactly and
 * the weights p are rounded to the operands' type before they meet V, so y
 * carries about one more rounding of that type than the formula: relative to
 * max_t |V_t|, at most 2^-8 (bf16), or 2^-11 and 2^-32 for each token seen
 * (f16, whose smallest numbers are 2^-31 of the largest weight), before y's own.
 * D = 64, 128 or 256; Hq a multiple of Hkv; pages*Hkv and width*page below 2^31;
 * every matrix 16-byte aligned.
 */
typedef struct abg_tree_attn_args {
    const void *q, *Kc, *Vc;
    const int32_t *table, *lens, *cu;
    const void *Kd, *Vd;
    const uint64_t *mask;
    const float *gate;
    void *y;
    float *ysum;
    int64_t B, N, Hq, Hkv, D, page, pages, width, drafts, words, max_span;
    int32_t type, y_type;
} abg_tree_attn_args;
/* Bytes of workspace; it depends on D, type, Hq/Hkv and max_span only (and on
 * the device). */
abg_status abg_tree_attn_workspace(int64_t Hq, int64_t Hkv, int64_t D, int64_t max_span, int type, int64_t *bytes);
abg_status abg_tree_attn(const abg_tree_attn_args *a, void *ws, int64_t ws_bytes, void *stream);
/* Failure-detection self-test: abg_tree_attn of 16-bit operands whose blocks
 * never bring copy `item` (0, 1, ..: K and V tiles in the order of their use),
 * so that waits run out after the 0.5 s limit in every block that has so many.
 * Both launches end, with bits 0 and 256 of the device status word set, no copy
 * or product in flight and the context usable; y holds no result.  A block
 * with fewer copies finishes its part. */
abg_status abg_selftest_tree_attn_timeout(const abg_tree_attn_args *a, void *ws, int64_t ws_bytes, int item,
                                          void *stream);

/*
 * tree_accept: the greedy check of the drafts.  best[n] is the index of the
 * largest of row n's V logits (the lowest such index; a NaN counts as
 * -infinity).  Draft 0 of a request is its last known token and is accepted;
 * from an accepted draft c the walk goes to the first later draft whose parent
 * is c and whose token is best[c], until there is none.
 *   logits f32, row n at logits + n*ld   tok, parent i32 [N] (as tree_plan's;
 *          a child comes after its parent)
 *   best   i32 [N]  (all N rows)
 *   rows   i32 [N]  rows[cu[b]+i] = row of the i-th accepted draft of request
 *          b (for abg_kv_put), -1 after the last and outside the spans
 *   add    i32 [B]  number of accepted drafts (for abg_page_plan)
 *   last   i32 [B]  best of the last accepted draft: the next token (-1 for an
 *          empty span)
 *   ws     abg_tree_accept_workspace() bytes, as tree_attn's
 * Drafts from ABG_MAX_SPAN on in a span are not accepted.
 */
abg_status abg_tree_accept_workspace(int64_t N, int64_t V, int64_t *bytes);
abg_status abg_tree_accept(const float *logits, int64_t ld, const int32_t *tok, const int32_t *parent,
                           const int32_t *cu, int32_t *best, int32_t *rows, int32_t *add, int32_t *last, int64_t B,
                           int64_t N, int64_t V, void *ws, int64_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Quantised cache: the paged cache of the draft-verification calls with its
 * rows in 4 or 8 bits, in the weights' format (value = scale*code + bias).
 *
 *   abg_kvq_put    rows into the cache, with kv_put's norm and rotation
 *   abg_kvq_attn   tree_attn over such a cache
 *   abg_kvq_get    rows of the cache read back
 *
 * They take the place of abg_kv_put and abg_tree_attn for the cache; the drafts
 * of a step stay in f32, bf16 or f16 rows.  Lengths, spans, tables, slots and
 * early starts are as there; the results are the same on every run.
 *
 * A row of D values of one head is D*bits/32 words and D/group factor pairs:
 *   Kc, Vc  u32 [pages][Hkv][page][D*bits/32]  codes, low first: code j of word
 *           k is column (32/bits)*k + j
 *   Ks, Vs  f16 [pages][Hkv][page][D/group][2]  scale, bias of each group
 * bits = 4 or 8, group = 32 or 64 columns, D = 64, 128 or 256, page >= 1, fewer than
 * 2^32 - 1 rows (pages*Hkv*page).
 * ------------------------------------------------------------------------- */
typedef struct abg_kvq_cache {
    void *Kc, *Ks, *Vc, *Vs;
    int64_t pages, Hkv, page, D;
    int32_t bits, group;
} abg_kvq_cache;

/*
 * kvq_put: key and value rows of N tokens into a quantised cache, k and q with
 * abg_atq's RMS norm and rotation (each optional).  Arguments as abg_kv_put's,
 * but src_type is any type, and qo is of q_type: src_type, or any type where
 * src_type is f32.
 *   Of the f32 values x of a group (normed and rotated in f32, not rounded to
 * 16 bits in between), each step rounded once to nearest even:
 *     bias  = f16(min x),  scale = f16((max x - min x) / (2^bits - 1)),
 *     code  = clamp(rint((x - bias) * (1 / scale)), 0, 2^bits - 1), 0 where
 *             scale is 0.
 *   A value is off by at most half a scale, the bias's rounding and 2^-11 of the
 * group's range (or (2^bits - 1)*2^-25, where the scale is below 2^-14).  A group
 * with a NaN or a magnitude above 65504 (f16's largest) is held as NaN: scale and
 * bias are 0x7fff, the codes 0.
 * The codes and factors are exact: they are the same on every run, and those of
 * these steps done one by one in any IEEE binary32 arithmetic (of zeros of both
 * signs -0 is the least).
 */
typedef struct abg_kvq_put_args {
    const void *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;
    const int32_t *rows;
    const int64_t *slots;
    const float *qn_w, *kn_w, *cos, *sin;
    const int32_t *pos;
    void *qo;
    abg_kvq_cache c;
    int64_t N, src_rows, Hq, cos_rows;
    float eps;
    int32_t src_type, q_type;
} abg_kvq_put_args;
abg_status abg_kvq_put(const abg_kvq_put_args *a, void *stream);

/*
 * kvq_get: the values of N rows of a quantised cache, scale*code + bias rounded
 * once to f32 and once more to `type`.
 *   k, v   row n, head h at k + n*k_row + h*k_head (in elements); each may be
 *          null (not both): then it is not read
 *   slots  i64 [N] or null: row n is slot slots[n] (null: n); a slot outside
 *          0 .. pages*page-1 gives zeros
 * Rows, row strides and head strides are multiples of 16 bytes; rows may not
 * lie in one another (k_row and k_head span distinct rows).
 * k and v may lie in one buffer, between one another's rows or heads: at the same
 * strides wherever no two rows meet (a single row's or head's stride does not
 * count), at others where whole rows or heads of the one lie between the other's.
 */
typedef struct abg_kvq_get_args {
    abg_kvq_cache c;
    const int64_t *slots;
    void *k, *v;
    int64_t k_row, k_head, v_row, v_head, N;
    int32_t type;
} abg_kvq_get_args;
abg_status abg_kvq_get(const abg_kvq_get_args *a, void *stream);

/*
 * kvq_attn: abg_tree_attn with the cached tokens' K and V in a quantised cache;
 * q, Kd and Vd of `type`, everything else as there.  One new token a request is
 * a span of 1.
 *   A page outside 0 .. pages-1 reads as zeros; a NaN in a K row that a query
 * sees makes its result NaN, one in a V row those columns' group (an infinite
 * factor, which kvq_put never writes, may do so too).  A row of q
 * that holds a NaN or a magnitude of 2^100 or more gives NaN (0 where it sees no
 * token).  width*page is at most 2^31 - 2048.
 *   Sums, softmax statistics and the work split's partial results are f32.
 * Codes are multiplied exactly, with q in f16 after a scaling of the row by a
 * power of two: 16-bit q as it is (elements below 2^-23 of the row's largest lose
 * bits), f32 q to 22 bits (of elements below 2^-12 of the largest: to 2^-34 of
 * that).  The weights p*scale that meet V's codes are rounded to 11 bits for
 * bf16 (whatever y's type), to 22 bits for f16 and f32, the smallest of either to
 * 2^-38 of the largest scale in V.  The tensor cores cut the sums of a block's products (up to
 * 32 tokens, 64 columns) off at about 2^-17 of the largest for bf16, at 2^-23 for
 * f16 and f32.  Drafts are multiplied in f32.
 *   The time grows with a request and head's rows (its span times Hq/Hkv): each 16
 * (8 at D = 256) go through the cache and its codes once more.  For bf16 and f16
 * queries it is shorter than abg_tree_attn's over the same rows in 16 bits up to 16
 * rows (8 at D = 256; 16 rows of f16 over 8 bits: as long) and longer from 32 on,
 * several times at 64 and more; for f32 ones it is a quarter to half of
 * abg_tree_attn's, and as much for a span of 256 over a few thousand tokens.
 * ws: abg_kvq_attn_workspace() bytes, as tree_attn's.
 */
typedef struct abg_kvq_attn_args {
    const void *q;
    abg_kvq_cache c;
    const int32_t *table, *lens, *cu;
    const void *Kd, *Vd;
    const uint64_t *mask;
    const float *gate;
    void *y;
    float *ysum;
    int64_t B, N, Hq, width, drafts, words, max_span;
    int32_t type, y_type;
} abg_kvq_attn_args;
/* Bytes of workspace; it depends on the cache's D, bits and group, type, Hq/Hkv
 * and max_span only (and on the device).  Pointers and pages of c are not read. */
abg_status abg_kvq_attn_workspace(const abg_kvq_cache *c, int64_t Hq, int64_t max_span, int type, int64_t *bytes);
abg_status abg_kvq_attn(const abg_kvq_attn_args *a, void *ws, int64_t ws_bytes, void *stream);

const char *abg_status_str(int status);
/* Text of the last CUDA error seen by any call on this thread ("" if none). */
const char *abg_last_cuda_error(void);

#ifdef __cplusplus
}
#endif
#endif /* ABG_H */
