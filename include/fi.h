/*
 * fi.h -- C-ABI of the MI355X exact autoregressive long-convolution library.
 *
 * What it computes.  Flash Inference (arXiv 2410.12982), summary page,
 * "Aufgabendefinition" and "LCSM-spezifische Definition": for every layer l,
 * batch row b and channel c, the mixer output at position n (1-based) is
 *
 *     y^l_n[b,c] = sum_{s=1..n} h^l[c][n-s] * x^l_s[b,c]
 *
 * where x^l_s is the layer's input at position s, which only becomes known
 * after position s-1 has been produced ("unlock y_{i+1}" in Algorithm 1).
 * The filters h^l are data independent and known ahead.
 *
 * How.  "Kachelung-Strategie (Algorithmus 1)" and "Schicht-uebergreifende
 * Parallelisierung (Algorithmus 3)": after position n the library adds the
 * contribution of inputs [n-U+1, n] to outputs [n+1, n+U], U = largest power
 * of two dividing n ("gray block"), for all layers in one batched launch; the
 * own-position term h^l[c][0] * x^l_n ("red cell") is added when position n is
 * produced.  A gray block is computed either directly or through an FFT of
 * length 2U against a cached filter spectrum ("Technische Innovationen",
 * "FFT-Vorberechnung" and "Zirkulaere Faltungs-Trick"), chosen per block size
 * ("Hybrid" in "Vergleichsmethoden"; selection by profiling per shape and
 * block size, rebuttal page).
 *
 * Conventions shared by every call.
 *  - Positions are 1-based; the context starts at position 0 (nothing
 *    produced).  L, the maximum number of positions, must be a power of two
 *    (so no gray block runs past L).
 *  - All device buffers are caller-owned plain device pointers (for example
 *    torch tensors' data pointers), fp32, row-major, densely packed.
 *  - All calls are ordered on the stream bound at fi_init and return without
 *    waiting for the device unless stated; outputs are valid once that stream
 *    has been synchronised.
 *  - Any HIP error poisons the context: that call and every later call except
 *    fi_destroy/fi_last_error/fi_position return FI_ESTATE (the failing call
 *    itself returns FI_EDEVICE).  fi_last_error() describes the first failure.
 *  - A context is not thread safe; use one context per stream.
 */
#ifndef FI_H
#define FI_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct fi_ctx fi_ctx; /* opaque, owned by the library */

typedef enum fi_status {
    FI_OK = 0,
    FI_EINVAL = -1,  /* bad argument (shape, null pointer, L not a power of two) */
    FI_ENOMEM = -2,  /* device memory could not be allocated / workspace too small */
    FI_EDEVICE = -3, /* a HIP call failed (the context is now poisoned) */
    FI_ERANGE = -4,  /* stepping past position L */
    FI_ESTATE = -5   /* context poisoned, or call not valid in the current mode */
} fi_status;

/* Map between layers: x^{l+1}_n = map(y^l_n).  Feedback: x^0_{n+1} = fb(y^{M-1}_n).
 * (The pages' synthetic model puts a block after each mixer and a sampler at
 * the end, "LCSM-Inferenz-Algorithmus"; the elementwise tanh stands in for both.)
 * FI_MAP_EXTERNAL: the caller runs its own block between layers with
 * fi_layer_red() / fi_tiles().
 * FI_MAP_HYENA: the library runs a Hyena-style block after every mixer
 * ("Modellarchitektur": a^l = block^l(mixer^l(a^{l-1}))), weights given by
 * fi_set_block_weights: [u|v|w] = x W, the mixer convolves q = u*w, its output
 * c gates m = v*c, z = GELU(m W1) W2 (exact-erf GELU, no biases),
 * a = z / sqrt(mean(z^2) + 1e-6), next layer input a, next position's layer-0
 * input fb(a^{M-1}).  Needs D % 8 == 0, D <= 768 and B <= 8.  Here "y" of fi_step /
 * fi_generate is a^{M-1}_n, the value the feedback is applied to. */
enum { FI_MAP_TANH = 0, FI_MAP_IDENTITY = 1, FI_MAP_EXTERNAL = 2, FI_MAP_HYENA = 3 };
enum { FI_FEEDBACK_TANH = 0, FI_FEEDBACK_IDENTITY = 1 };

/* How gray blocks are computed. AUTO: per block size, the faster path as timed
 * on the device at fi_init; DIRECT/FFT force one path where it exists (direct
 * blocks exist for U <= 128, FFT blocks for U >= 4). */
enum { FI_TAU_AUTO = 0, FI_TAU_DIRECT = 1, FI_TAU_FFT = 2 };
enum { FI_PATH_NONE = 0, FI_PATH_DIRECT = 1, FI_PATH_FFT = 2 };

typedef struct fi_options {
    int map;               /* FI_MAP_*; default FI_MAP_TANH */
    int feedback;          /* FI_FEEDBACK_*; default FI_FEEDBACK_TANH */
    int tau_mode;          /* FI_TAU_*; default FI_TAU_AUTO */
    int tau_split;         /* -1: per-class choice (AUTO calibrates); q >= 0: classes
                              with U = 2^q' >= 2^q use FFT, smaller ones DIRECT */
    int record;            /* 1: keep every layer's input and mixer output (tests) */
    int use_graphs;        /* 1 (default): fi_generate replays captured hipGraphs */
    int block_graph_log2;  /* k: a block graph replays the 2^k - 1 positions between
                              multiples of 2^k (default 6; 0 disables) */
    int filters_on_device; /* 1: the filters pointer given to fi_init is device memory */
    int fft_max_log2;      /* widest gray block done as one workgroup transform, as
                              log2(U) in [12, 14] (default 14: 128 KB of LDS); the
                              next class runs as two halves of that width in one
                              workgroup, wider blocks are split into sub-blocks of
                              that width */
    int time_blocks;       /* 1: fi_generate brackets every FFT gray-block launch with
                              HIP events stamped by the launches themselves (read with
                              fi_block_times); those positions then bypass graphs */
    int defer_wide;        /* 1: a split gray block at position n computes only its
                              first output sub-block (V positions) before position
                              n+1; the others run on a second stream of the context,
                              overlapping positions n+1 .. n+V-1, and the context
                              stream waits for them before position n+V.  Cuts the
                              latency of that position; results are bit for bit
                              those without it.  2: the same, and the two-half
                              class (twice fft_max_log2) is deferred too, run as 4
                              sub-blocks of half the one-workgroup width (V =
                              2^(fft_max_log2-1)); its results then differ from the
                              two-half kernel's by rounding.  Level 2 needs
                              fft_max_log2 >= 13, adds the offset spectra of that
                              width to the workspace (7 * V/2 float4 per (l, c)),
                              and where no two-half class exists acts as 1.
                              Default 0 */
    int chunk_direct;      /* 1 (default): for maps that act channel by channel
                              (FI_MAP_TANH, FI_MAP_IDENTITY), fi_generate and
                              fi_prefill run the G = 2^q positions between two
                              FFT positions (q: the first FFT class) as one
                              launch, each workgroup owning whole chains.  The
                              direct gray blocks of a chunk then sum, target by
                              target, the same pairs the tiling assigns them
                              (summary page, "Kachelung-Strategie"; the blocks
                              below G never leave a chunk).  0: one launch (or
                              graph node) per position */
    int eager_prefill;     /* 1 (default): fi_prefill at position 0 computes the
                              prompt layer by layer with all of a layer's
                              positions at once (direct sums inside blocks of G,
                              FFT blocks above), when the map acts channel by
                              channel, P is a multiple of G, P <= L/2, and every
                              gray block after n <= P wider than one workgroup
                              transform either starts at n = P or (the two-half
                              class) ends inside the prompt -- e.g. at
                              L = 2^17, P = 16384, 32768, 65536 -- otherwise, or
                              with 0, P teacher-forced positions */
    int reserved[3];       /* must be zero */
} fi_options;

/* Fill *opt with the defaults listed above. */
void fi_default_options(fi_options *opt);

/* Library version string, e.g. "fi 0.1 gfx950". */
const char *fi_version(void);

/* Device bytes fi_init needs for this shape and options (0 on bad arguments).
 * The workspace holds the filters, the per-layer activation rows (inputs for
 * positions <= n, pending sums for positions > n: the pages' activation reuse,
 * "Speicheroptimierung"), the cached filter spectra and scratch. */
size_t fi_workspace_bytes(int layers, int batch, int channels, int64_t L,
                          const fi_options *opt);

/* Create a context.
 *   layers M >= 1, batch B >= 1, channels D >= 1, L = 2^P with 1 <= L <= 2^24.
 *   filters: fp32 [M][D][L] (layer-major, channel rows of L taps h[0..L-1]),
 *            host memory unless opt->filters_on_device; copied, the caller keeps
 *            ownership and may free it when fi_init returns.
 *   opt:     NULL for defaults.
 *   workspace: device buffer of at least fi_workspace_bytes() bytes, 256-byte
 *            aligned, owned by the caller and untouched by it while the context
 *            lives; or NULL to let the library allocate (and free) its own.
 *   stream:  hipStream_t the context runs on (NULL = default stream).
 * Computes the filter spectra and, for FI_TAU_AUTO, times the block paths on
 * the device: with chunked positions (fi_options.chunk_direct and a map that
 * acts channel by channel), one chunk plus its FFT block per candidate split
 * (fi_chunk_table); otherwise both paths per block size (fi_tau_table).
 * Synchronises the stream before returning.
 * Returns FI_EINVAL / FI_ENOMEM / FI_EDEVICE on failure (*out is then NULL). */
fi_status fi_init(fi_ctx **out, int layers, int batch, int channels, int64_t L,
                  const float *filters, const fi_options *opt, void *workspace,
                  void *stream);

/* Release the context (and its own allocations).  Safe on NULL. */
fi_status fi_destroy(fi_ctx *ctx);

/* Back to position 0 with all activations cleared; filters, spectra and the
 * block-path table are kept. */
fi_status fi_reset(fi_ctx *ctx);

/* Set fi_options.defer_wide (0, 1 or 2) for the following positions.
 * Large-block latency (Flash Inference summary page, "Hauptergebnisse": the
 * per-token time spikes at the positions of the widest blocks): with it on, a
 * split gray block (level 2: also a two-half block) puts its later output
 * sub-blocks on the context's second stream.  Any deferred work still running
 * is joined into the context stream first.  FI_EINVAL for other values;
 * FI_ESTATE for 2 when the context has a two-half class that fi_init did not
 * prepare (fi_options.defer_wide was not 2 there). */
fi_status fi_set_defer_wide(fi_ctx *ctx, int on);

/* Produce the next position n = fi_position()+1 (Algorithm 2 for one i).
 *   x_t: device fp32 [B][D], the layer-0 input x^0_n; NULL = feedback
 *        (x^0_n = fb(y^{M-1}_{n-1}); at n = 1 the value given by fi_set_input).
 *   y_t: device fp32 [B][D] receiving the last layer's mixer output
 *        y^{M-1}_n (before the map), or NULL.
 * Runs the red cells of all layers in order, then the gray blocks of all
 * layers after n.  FI_ERANGE when the position is already L.
 * Not valid in FI_MAP_EXTERNAL mode (FI_ESTATE). */
fi_status fi_step(fi_ctx *ctx, const float *x_t, float *y_t);

/* Set the layer-0 input used by the next feedback step when no previous
 * output exists (position 0), device fp32 [B][D]. */
fi_status fi_set_input(fi_ctx *ctx, const float *x0);

/* Teacher-forced prompt (Flash Inference rebuttal page, reply on prefill: the
 * prompt is given at once, so its contributions to all later outputs can be
 * pushed eagerly; summary page, "Einschraenkungen": prefill dominates the
 * cost for long prompts): equivalent to P calls fi_step(x + (i-1)*B*D, y ...)
 * for i = 1..P (the invariant the tests check).
 *   x: device fp32 [P][B][D]; y: device fp32 [P][B][D] or NULL.
 * The prompt's positions are processed in place (position advances by P). */
fi_status fi_prefill(fi_ctx *ctx, const float *x, int64_t P, float *y);

/* Free-running generation of `steps` positions with internal feedback (summary
 * page, "LCSM-Inferenz-Algorithmus", Algorithm 2: per position the layers' red
 * cells in order, the next input from the last layer's output, then every
 * layer's gray block; "Schicht-uebergreifende Parallelisierung", Algorithm 3:
 * the gray blocks of all layers in one launch), with one hipGraph per
 * block-size class plus block graphs (use_graphs = 1) or chunk launches.
 *   y: device fp32 [steps][B][D] receiving y^{M-1}_n for each position, or NULL.
 * FI_ERANGE if position + steps > L (nothing is run). */
fi_status fi_generate(fi_ctx *ctx, int64_t steps, float *y);

/* Positions produced so far (0..L). */
int64_t fi_position(const fi_ctx *ctx);

/* Human-readable description of the first failure, or "" . */
const char *fi_last_error(const fi_ctx *ctx);

/* Schedule of step n (1 <= n <= L): *q = log2 of the gray-block edge after n
 * (or -1 for n = L, which has no gray block); *path = FI_PATH_* used for it. */
fi_status fi_debug_schedule(const fi_ctx *ctx, int64_t n, int *q, int *path);

/* Block-path table: for q = 0..P-1 writes path[q] (FI_PATH_*) and, when
 * calibration ran, the measured microseconds per launch of the direct and FFT
 * paths (negative where a path does not exist or was not timed).  Arrays hold
 * at least P entries; any pointer may be NULL. */
fi_status fi_tau_table(const fi_ctx *ctx, int *path, double *us_direct, double *us_fft);

/* Chunk-path calibration (FI_TAU_AUTO with chunked positions): for each
 * candidate first FFT class g (chunks of 2^g positions carry every block below
 * 2^g), us_chunk[g] = measured microseconds of one chunk and the class-g FFT
 * gray blocks after it, us_run[g] = the modeled microseconds of the classes
 * the choice affects over a whole run ((L / 2^g) chunks plus the FFT blocks of
 * classes g .. 8); the split used is the shortest chunk whose us_run is within
 * 1.5% of the least (closer than the timing repeats), so repeated
 * calibrations agree.  -1 where not timed.  Arrays hold at least P + 1 entries; either may be NULL. */
fi_status fi_chunk_table(const fi_ctx *ctx, double *us_chunk, double *us_run);

/* Copy positions first..first+count-1 (first >= 1) of one layer into dst
 * (device fp32, [count][B][D]):
 * what = 0: the layer's convolution inputs x^l_s, what = 1: its mixer outputs
 * y^l_s, what = 2 (FI_MAP_HYENA only): its block outputs a^l_s (valid for
 * s <= position).  Needs record = 1 (FI_ESTATE otherwise). */
fi_status fi_history(const fi_ctx *ctx, int layer, int what, int64_t first, int64_t count, float *dst);

/* Block weights for FI_MAP_HYENA, as bf16 bit patterns in row-major x*W
 * layout: W [M][D][3D], W1 [M][D][4D], W2 [M][4D][D]; host memory unless
 * on_device.  Copied (stored transposed); the caller keeps ownership.
 * Synchronises the stream.  Must precede any step in that mode (FI_ESTATE). */
fi_status fi_set_block_weights(fi_ctx *ctx, const uint16_t *W, const uint16_t *W1, const uint16_t *W2,
                               int on_device);

/* fi_set_block_weights for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same upload and the same result, but the staging buffer the
 * weights pass through on their way to the transposed layout is a fixed
 * device array of the library (4.5 MiB per device, its address looked up at
 * the first call on a device) instead of an allocation; no hipMalloc, hipFree
 * or other allocating call is made.  Limit: 4*D*D 16-bit values must fit the
 * array, i.e. D <= 768, the widest block FI_MAP_HYENA takes (FI_EINVAL with a
 * message otherwise).  Every call on one device shares that device's array
 * and leaves its contents there: calls that overlap on one device (other
 * streams or threads) race.  Synchronises the stream, like
 * fi_set_block_weights. */
fi_status fi_set_block_weights_static(fi_ctx *ctx, const uint16_t *W, const uint16_t *W1, const uint16_t *W2,
                                      int on_device);

/* Device wall-clock stamps (100 MHz counter ticks) written when each position
 * finished: dst (host int64 [count]) receives the stamps of positions
 * first..first+count-1.  Synchronises the stream. */
fi_status fi_stamps(fi_ctx *ctx, int64_t first, int64_t count, int64_t *dst);

/* External-block mode (FI_MAP_EXTERNAL).  For the current position
 * n = fi_position()+1 the caller, for l = 0..M-1 in order, supplies the
 * layer's mixer input q (device [B][D]) and receives its mixer output
 *     y^l_n = (pending sum at n) + h^l[c][0] * q
 * (the red cell of Algorithm 2), then calls fi_tiles() to run all layers'
 * gray blocks after n and advance to n.  y may alias nothing else. */
fi_status fi_layer_red(fi_ctx *ctx, int layer, const float *q, float *y);
fi_status fi_tiles(fi_ctx *ctx);

/* GPU Lazy baseline ("Vergleichsmethoden", Lazy: each position computes its
 * full sum on demand, O(n) per position, all layers' sums in parallel):
 * same semantics as fi_step / fi_generate (internal feedback) on a context
 * that has not run any tiled step since fi_init/fi_reset (FI_ESTATE
 * otherwise; likewise tiled calls after Lazy calls until fi_reset). */
fi_status fi_lazy_step(fi_ctx *ctx, const float *x_t, float *y_t);
fi_status fi_lazy_generate(fi_ctx *ctx, int64_t steps, float *y);

/* The pages' baselines and their ablations ("Vergleichsmethoden": Lazy,
 * Eager, Lazy NP, Eager NP; "Ablationsstudien", cross-layer parallelism):
 *   FI_BASE_LAZY      position n computes its full O(n) sum, all layers in
 *                     one launch, then the red cells (= fi_lazy_step);
 *   FI_BASE_EAGER     the red cells of n, then x_n is pushed into the pending
 *                     sums of every later position (O(L - n)), all layers in
 *                     one launch;
 *   FI_BASE_LAZY_NP,
 *   FI_BASE_EAGER_NP  the same with the per-row work launched layer by layer
 *                     (no cross-layer parallelism).
 * fi_baseline_step / fi_baseline_generate have the semantics of fi_step /
 * fi_generate (x_t device [B][D] or NULL for internal feedback; y_t device
 * [B][D] or NULL; y device [steps][B][D] or NULL).  A context steps one
 * family at a time: Lazy kinds and Eager kinds, and either with tiled calls,
 * cannot be mixed without fi_reset (FI_ESTATE).  kind outside the list:
 * FI_EINVAL; external-block and Hyena-style maps: FI_ESTATE. */
enum { FI_BASE_LAZY = 0, FI_BASE_EAGER = 1, FI_BASE_LAZY_NP = 2, FI_BASE_EAGER_NP = 3 };
fi_status fi_baseline_step(fi_ctx *ctx, int kind, const float *x_t, float *y_t);
fi_status fi_baseline_generate(fi_ctx *ctx, int kind, int64_t steps, float *y);

/* Benchmark support for the baselines: the mean device time in microseconds
 * of one baseline position n of the given kind (its sums or pushes plus the
 * red cells), over `reps` launches timed with HIP events, without advancing.
 * Overwrites activation rows: fi_reset is required before further stepping
 * (FI_ESTATE otherwise). */
fi_status fi_baseline_time(fi_ctx *ctx, int kind, int64_t n, int reps, double *us);

/* Per-class FFT gray-block timing (needs time_blocks = 1): for q = 0..P-1,
 * ms[q] = summed event-measured milliseconds of the FFT gray-block kernels of
 * class q launched by fi_generate, count[q] = number of such launches.
 * Synchronises the stream.  clear = 1 zeroes the sums afterwards.  Arrays hold
 * at least P entries; either may be NULL. */
fi_status fi_block_times(fi_ctx *ctx, int clear, double *ms, int64_t *count);

/* Chunk-kernel timing (needs time_blocks = 1): *ms = summed event-measured
 * milliseconds of the chunk kernels fi_generate / fi_step launched (each runs
 * the red cells and direct gray blocks of 2^k consecutive positions, see
 * fi_options.chunk_direct), *count = their number.  Synchronises the stream;
 * clear = 1 zeroes both afterwards.  Either pointer may be NULL. */
fi_status fi_chunk_times(fi_ctx *ctx, int clear, double *ms, int64_t *count);

/* Per-size runtime of one gray-block path (the pages' runtime-per-tile-size
 * comparison, "Pareto-Optimalitaetskurve"): the mean device time in
 * microseconds of the gray-block kernels of class q (U = 2^q) over `reps`
 * launches at position n = 2^q, timed with HIP events, without advancing.
 * path = FI_PATH_DIRECT (the direct kernel, red cells included) or
 * FI_PATH_FFT (the FFT kernels alone).  FI_EINVAL where the path does not
 * exist for q.  Overwrites activation rows: fi_reset is required before any
 * further stepping (FI_ESTATE otherwise). */
fi_status fi_time_block(fi_ctx *ctx, int q, int path, int reps, double *us);

/* Benchmark support for the time split between mixer and block (summary page,
 * "Zeit-Zerlegung (Abbildung 2a)"): the mean device time in microseconds of
 * one position's block kernels in FI_MAP_HYENA mode -- every layer's
 * projection (with its red cell), GELU up-projection and down-projection, then
 * the RMSNorm'd output and feedback -- without the gray blocks, over `reps`
 * launches timed with HIP events, without advancing.  Needs the block weights
 * (FI_ESTATE otherwise).  The activation rows are overwritten: fi_reset is
 * required before any further stepping (FI_ESTATE otherwise). */
fi_status fi_time_hyena_block(fi_ctx *ctx, int reps, double *us);

/* Benchmark support for the Lazy baseline: the mean device time in
 * microseconds of the Lazy work of position n (every layer's full O(n) sum
 * plus the red cells), over `reps` launches timed with HIP events, without
 * advancing.  The activation rows are overwritten: the context must be reset
 * (fi_reset) before any further stepping (FI_ESTATE otherwise). */
fi_status fi_lazy_time(fi_ctx *ctx, int64_t n, int reps, double *us);

/* ------------------------------------------------------------------------
 * Data-dependent filters.  Flash Inference, summary page, "Datenabhaengige
 * Filter-Erweiterung (Appendix B)": with a filter that depends on the data, a
 * modified tiling (Algorithm 5) keeps the method exact at twice the work; the
 * rebuttal page adds that each block then takes two same-size transforms
 * instead of one.  The pages give nothing more.  Reading used here: both
 * sequences arrive online, per batch row b and channel c the input x_t and the
 * filter tap h_t at position t (0-based, t = 0 .. L-1), and
 *
 *     y_t[b,c] = sum_{i+j=t} x_i[b,c] * h_j[b,c]
 *
 * (one layer; taps per (b, c), since a data-dependent filter differs per
 * sequence).  Tiling, p a power of two: red cell y_t = pend_t + x_t h_0 +
 * x_0 h_t; at t = 2p-1 the square x[p, 2p) * h[p, 2p); at t = (m+1)p-1,
 * m >= 2, the two band products x[t+1-p, t] * h[p, 2p) and h[t+1-p, t] *
 * x[p, 2p).  Each adds into the pending sums of positions t+1 .. t+2p-1.
 * Products of p >= 2^fft_min_log2 run as 2p-point FFTs against the cached
 * spectrum of the fixed block, smaller ones directly.
 *
 * One context per stream; calls are stream-ordered on the bound stream and
 * not thread-safe.  All pointers are caller-owned device memory, fp32,
 * [B][D] per position (row r = b*D + c), densely packed.
 * ------------------------------------------------------------------------ */
typedef struct fi_dd fi_dd; /* opaque, owned by the library */

/* Device bytes the workspace of a data-dependent context needs: three
 * [B*D][L] fp32 arrays (inputs, taps, pending sums) plus the fixed-block
 * spectra (16 L bytes per row), twiddles and one [B*D] array (the layer
 * inputs of a position, used by stacks).  0 if the shape is unsupported:
 * B, D >= 1, B*D <= 2^24, L a power of two up to 32768 (the widest product,
 * L/2 points, must fit one workgroup's transform); fft_min_log2 in [2, 15], or
 * -1 for the default 8.  Products of p < 2^fft_min_log2 run directly: up to
 * p = 128 inside the position's first launch (one thread per target), wider
 * ones one thread per row; the rest as FFTs. */
size_t fi_dd_workspace_bytes(int batch, int channels, int64_t L, int fft_min_log2);

/* Create a context at position 0 over the caller's workspace (device, at
 * least fi_dd_workspace_bytes, 256-byte aligned; the context keeps using it
 * until fi_dd_destroy).  stream: the hipStream_t every call of the context is
 * ordered on (NULL = default stream).  Synchronises the stream.  FI_EINVAL for a null
 * pointer or an unsupported shape, FI_EDEVICE if a HIP call fails. */
fi_status fi_dd_init(fi_dd **out, int batch, int channels, int64_t L, int fft_min_log2, void *workspace,
                     void *stream);

/* A stack of `layers` data-dependent layers in one context (the summary page's
 * layer stacks, "Schicht-uebergreifende Parallelisierung (Algorithmus 3)",
 * with the filters of "Datenabhaengige Filter-Erweiterung (Appendix B)"):
 * at each position layer l's taps h^l_t arrive with the data, layer 0's input
 * x^0_t too, and layer l+1's input is tanh(y^l_t).  The red cells run layer
 * after layer (one thread per (b, c) chain); every product of the position
 * then runs once for the rows of all layers.  Sizes and limits as
 * fi_dd_workspace_bytes, with 1 <= layers <= 64 and layers * batch * channels
 * rows; 0 for an unsupported shape. */
size_t fi_dd_stack_workspace_bytes(int layers, int batch, int channels, int64_t L, int fft_min_log2);

/* Create a stack context (as fi_dd_init; layers = 1 is the single layer). */
fi_status fi_dd_stack_init(fi_dd **out, int layers, int batch, int channels, int64_t L, int fft_min_log2,
                           void *workspace, void *stream);

/* One position: x_t ([B][D], device: layer 0's input) and h_t ([M][B][D],
 * device: every layer's tap, M the context's layers, 1 for fi_dd_init) arrive,
 * y_t ([M][B][D], device: every layer's output) is written.  FI_ERANGE after
 * L positions, FI_EINVAL for null pointers, FI_ESTATE after a device failure. */
fi_status fi_dd_step(fi_dd *ctx, const float *x_t, const float *h_t, float *y_t);

/* `steps` positions in a row: x is [steps][B][D], h and y [steps][M][B][D]
 * (device). */
fi_status fi_dd_run(fi_dd *ctx, const float *x, const float *h, int64_t steps, float *y);

/* Back to position 0 (inputs, taps and pending sums cleared). */
fi_status fi_dd_reset(fi_dd *ctx);

/* Positions produced so far (-1 for a null context). */
int64_t fi_dd_position(const fi_dd *ctx);

/* Message of the last failed call. */
const char *fi_dd_last_error(const fi_dd *ctx);

/* Synchronise the stream and free the context (not the workspace); FI_OK
 * for a null context, FI_EDEVICE if the synchronisation fails. */
fi_status fi_dd_destroy(fi_dd *ctx);

/* ------------------------------------------------------------------------
 * Operators of a recurrent block: what a caller that runs its own block
 * between mixers (FI_MAP_EXTERNAL, fi_layer_red / fi_tiles) or trains one
 * needs next to the long convolution.  They hold no context: every call takes
 * its sizes, device pointers and stream, allocates nothing, waits for nothing
 * and may be captured into a graph.
 *
 * Conventions shared by these calls.
 *  - Tensors are row-major; a row is `channels` contiguous values and rows are
 *    a pitch (ld_*, in elements, 0 = densely packed) apart, so a tensor may be
 *    a column slice of a wider one.  Sequences are [T][B][D]: row t*B + b.
 *  - Types: FI_F32, FI_BF16, FI_F16.  Arithmetic, states, sums and statistics
 *    are fp32; a value is rounded once, when it is stored.
 *  - An output may not share an element with an input or another output,
 *    unless stated (FI_EINVAL); column slices of one tensor are separate.
 *  - A workspace (256-byte aligned) belongs to one call until its work on the
 *    stream is done; its contents need no initialisation and do not survive.
 *  - Pointers are aligned to their values, workspaces, saved states and packed
 *    weights to 256 bytes.
 *  - FI_EINVAL for a bad argument, FI_EDEVICE for a failed launch; nothing is
 *    launched when FI_EINVAL is returned.  fi_op_last_error() describes the
 *    calling thread's last failure.
 * ------------------------------------------------------------------------ */
enum { FI_F32 = 0, FI_BF16 = 1, FI_F16 = 2 };

/* Message of the calling thread's last failed operator call ("" if none). */
const char *fi_op_last_error(void);

/* The gated linear recurrence, per batch row b and channel c:
 *
 *     z_t = gate_t + bias[c],  d_t = 1 - sigmoid(z_t)  (the decay's complement),
 *     s_t = (1 - d_t) s_{t-1} + e(d_t) x_t,            y_t = s_t,
 *
 * with the input factor e = 1 (PLAIN), d (CONVEX: a running average) or
 * sqrt(d (2 - d)) (ENERGY: keeps the variance of independent inputs). */
enum { FI_SCAN_PLAIN = 0, FI_SCAN_CONVEX = 1, FI_SCAN_ENERGY = 2 };

typedef struct fi_scan_desc {
    int64_t T;             /* positions, 0 .. 2^23 */
    int batch, channels;   /* B, D >= 1, B * D <= 2^24, ceil(T / 256) * B * D <= 2^28 (D < 4: 2^26) */
    int dtype;             /* of x, gate, y and their gradients */
    int input;             /* FI_SCAN_* */
    int64_t ld_x, ld_gate, ld_y;            /* row pitches, elements; 0 = channels */
    int64_t ld_dy, ld_dx, ld_dgate;
    int reserved[4];       /* must be zero */
} fi_scan_desc;

/* Bytes of the states the forward pass keeps for the backward pass (`saved`),
 * and of the workspace of either pass; 0 for a bad descriptor.  256 for the
 * forward pass means that its workspace is not used and may be NULL; the
 * backward pass needs one at every T > 0. */
size_t fi_scan_saved_bytes(const fi_scan_desc *desc);
size_t fi_scan_workspace_bytes(const fi_scan_desc *desc, int backward);

/* y [T][B][D] and, where not NULL, final [B][D] fp32 (the state after the last
 * position) and saved (for fi_scan_backward).  bias [D] fp32 or NULL (zeros);
 * state [B][D] fp32, the state before the first position, or NULL (zeros);
 * lengths [B] int32 (device) or NULL: row b has positions t < lengths[b] (taken
 * into [0, T]); what later rows hold counts for nothing, they give y = 0 and
 * leave the state as it is.  final may be state.  T = 1 is the form for one token:
 * one launch.  Of the positions that count, an infinity or NaN in x or the state,
 * or a NaN in gate, makes its channel's later values non-finite (from an infinity,
 * NaN may come one position on); an infinite gate is a decay of exactly 0 or 1.
 * A long sequence runs in tiles that hand the state on.  A tile that has waited
 * for the one before it through 2^20 looks (about a second: the launch is not
 * running as it should) goes on with NaN; the call has returned FI_OK by then. */
fi_status fi_scan_forward(const fi_scan_desc *desc, const void *x, const void *gate, const float *bias,
                          const float *state, const int32_t *lengths, void *y, float *final, void *saved,
                          void *workspace, void *stream);

/* Gradients of sum(y . dy) + sum(final . dfinal): dx, dgate [T][B][D] (0 past a
 * row's length), and where not NULL dbias [D] fp32 (summed over t and b in a
 * fixed order) and dstate [B][D] fp32.  The other arguments are those of the
 * forward call that wrote `saved`; dfinal may be NULL (zeros).  Tiles wait as in
 * the forward pass. */
fi_status fi_scan_backward(const fi_scan_desc *desc, const void *x, const void *gate, const float *bias,
                           const float *state, const int32_t *lengths, const void *saved, const void *dy,
                           const float *dfinal, void *dx, void *dgate, float *dbias, float *dstate,
                           void *workspace, void *stream);

/* The gated delta rule: a recurrence whose state is a matrix S [dk][dv], per batch
 * row and head:
 *
 *     S_t = a_t (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,  a_t = e^decay_t,
 *     y_t = scale S_t^T q_t
 *
 * with the write strength b = beta (0 .. 1, or to 2 for a map with negative
 * eigenvalues).  With `unit`, k and q are divided by their lengths first: k /
 * sqrt(sum k^2 + 10^-6); without, keys of about length one are the caller's (a map
 * of norm over one grows without end).  Groups of heads / key_heads heads share a
 * query and key head: head h takes the key head h / (heads / key_heads). */
typedef struct fi_delta_desc {
    int64_t T;             /* positions, 0 .. 2^23 */
    int batch;             /* B >= 1 */
    int key_heads, heads;  /* HK, H >= 1, H a multiple of HK, B H <= 2^20, and less than 2^24
                              with the chunks of T: of 64 positions, 32 for FI_F16 and FI_F32 */
    int dk, dv;            /* 1 .. 128, 1 .. 1024 */
    int dtype;             /* of q, k, v, y and their gradients */
    int unit;              /* 0 or 1 */
    float scale;
    int64_t ld_q, ld_k, ld_v, ld_decay, ld_beta, ld_y;   /* row pitches, elements; 0 = a row's own length; B rows at most 2^24 */
    int64_t ld_dy, ld_dq, ld_dk, ld_dv, ld_ddecay, ld_dbeta;
    int reserved[4];       /* must be zero */
} fi_delta_desc;

/* Bytes of what the forward pass keeps for the backward pass (`saved`), and of the
 * workspace of either pass; 0 for a bad descriptor.  A forward call of up to 14
 * positions that saves nothing uses no workspace (it may be NULL). */
size_t fi_delta_saved_bytes(const fi_delta_desc *desc);
size_t fi_delta_workspace_bytes(const fi_delta_desc *desc, int backward);

/* q, k [T][B][HK][dk], v [T][B][H][dv], decay and beta [T][B][H] fp32; state
 * [B][H][dk][dv] fp32, the state before the first position, or NULL (zeros);
 * lengths as in fi_scan_forward.  y [T][B][H][dv] (0 past a row's length) and,
 * where not NULL, final [B][H][dk][dv] fp32 (it may be state) and saved.
 * A decay of -infinity (any below -10^4) forgets everything before its position.
 * Products are of fp32 quality (three bf16 terms a factor), also those that only a
 * 16-bit y is made of.  Values, sums of squares and products of keys and queries
 * stay below 2^127; of factors below 2^-110 the last terms may be lost.  An infinity
 * or NaN in the state, or at a position that counts, makes its head's values
 * non-finite from the start of its chunk on (64 positions, 32 for FI_F16 and
 * FI_F32); other heads and rows are as without it. */
fi_status fi_delta_forward(const fi_delta_desc *desc, const void *q, const void *k, const void *v, const float *decay,
                           const float *beta, const float *state, const int32_t *lengths, void *y, float *final,
                           void *saved, void *workspace, void *stream);

/* Gradients of sum(y . dy) + sum(final . dfinal): dq, dk, dv per row (dq and dk
 * summed over the heads that share them), ddecay and dbeta [T][B][H] fp32, all 0
 * past a row's length, and where not NULL dstate [B][H][dk][dv] fp32.  The other
 * arguments are those of the forward call that wrote `saved`; dfinal may be NULL
 * (zeros).  A decay's gradient is summed of terms that carry the decay, so it keeps
 * its digits however small it makes them (0 at -infinity). */
fi_status fi_delta_backward(const fi_delta_desc *desc, const void *q, const void *k, const void *v, const float *decay,
                            const float *beta, const float *state, const int32_t *lengths, const void *saved,
                            const void *dy, const float *dfinal, void *dq, void *dk, void *dv, float *ddecay,
                            float *dbeta, float *dstate, void *workspace, void *stream);

/* The norms around a block, with the block's gate, residual and residual scale,
 * per row of `channels` values (each factor that is NULL is left out):
 *
 *     v = post_norm ? o / sqrt(mean(o^2) + eps) * post_weight : o
 *     m = v * act(gate)            act: FI_GATE_LINEAR, _SIGMOID, _SILU
 *     r = res + scale * m          the residual stream after the block
 *     a = r / sqrt(mean(r^2) + eps) * pre_weight     the next block's input
 *
 * o NULL (then gate, scale and post_norm are too): r = res, the norm before a
 * first block.  post_weight needs post_norm.  The mean is over the row; a
 * row whose squares' sum passes fp32's largest number is normed to 0.  a is
 * formed from r before r is rounded. */
enum { FI_GATE_LINEAR = 0, FI_GATE_SIGMOID = 1, FI_GATE_SILU = 2 };

typedef struct fi_norm_desc {
    int64_t rows;          /* >= 0 */
    int channels;          /* 1 .. 16384 */
    int dtype;             /* of o, gate, a and their gradients */
    int res_dtype;         /* of res, r and their gradients: dtype or FI_F32 */
    int post_norm;         /* 0 or 1 */
    int act;               /* FI_GATE_*, used where gate is given */
    float eps;             /* >= 0 */
    int64_t ld_o, ld_gate, ld_res, ld_r, ld_a;   /* row pitches, elements; 0 = channels */
    int64_t ld_dr, ld_da, ld_do, ld_dgate, ld_dres;
    int reserved[4];       /* must be zero */
} fi_norm_desc;

/* Workspace of fi_norm_backward; 0 for a bad descriptor. */
size_t fi_norm_workspace_bytes(const fi_norm_desc *desc);

/* r and a (either may be NULL), and where not NULL saved [2][rows] fp32 (the
 * two reciprocal norms, for the backward pass).  Weights and scale are fp32
 * [channels] or NULL.  r may be res itself (same pointer and pitch). */
fi_status fi_norm_forward(const fi_norm_desc *desc, const void *o, const void *gate, const void *res,
                          const float *post_weight, const float *scale, const float *pre_weight, void *r, void *a,
                          float *saved, void *stream);

/* Gradients of sum(r . dr) + sum(a . da) (dr or da may be NULL: zeros): where
 * not NULL d_o, dgate, dres per row and dpost, dscale, dpre fp32 [channels]
 * (summed over the rows in a fixed order).  A gradient can be asked for only
 * where its input is given, except that unit weights have gradients too: dpost
 * needs post_norm, dscale needs o, dpre needs da.  dres may be dr itself. */
fi_status fi_norm_backward(const fi_norm_desc *desc, const void *o, const void *gate, const void *res,
                           const float *post_weight, const float *scale, const float *pre_weight, const float *saved,
                           const void *dr, const void *da, void *d_o, void *dgate, void *dres, float *dpost,
                           float *dscale, float *dpre, void *workspace, void *stream);

/* The layer norm with a residual, per row of `channels` values:
 *
 *     r = res + x
 *     a = (r - mean(r)) / sqrt(mean((r - mean(r))^2) + eps) * weight + bias
 *
 * x or res may be NULL (not both: r is the other; with x NULL, a is of dtype and
 * res of res_dtype, so an fp32 stream is normed into 16 bits), weight and bias
 * too (1 and 0).  The means are over the row.  A row whose deviations' squares
 * pass fp32's largest number is normed to 0, one whose sum does gives NaN; the
 * other rows are as they would be without it.  a is formed from r before r is
 * rounded. */
typedef struct fi_layer_desc {
    int64_t rows;          /* >= 0 */
    int channels;          /* 1 .. 16384 */
    int dtype;             /* of x, a and their gradients */
    int res_dtype;         /* of res, r and their gradients: dtype or FI_F32 */
    float eps;             /* >= 0 */
    int64_t ld_x, ld_res, ld_r, ld_a;            /* row pitches, elements; 0 = channels */
    int64_t ld_dr, ld_da, ld_dx, ld_dres;
    int reserved[4];       /* must be zero */
} fi_layer_desc;

/* Workspace of fi_layer_backward; 0 for a bad descriptor. */
size_t fi_layer_workspace_bytes(const fi_layer_desc *desc);

/* r and a (either may be NULL), and where not NULL saved [2][rows] fp32 (mean
 * and reciprocal deviation, for the backward pass).  weight and bias are fp32
 * [channels].  r may be res itself (same pointer and pitch). */
fi_status fi_layer_forward(const fi_layer_desc *desc, const void *x, const void *res, const float *weight,
                           const float *bias, void *r, void *a, float *saved, void *stream);

/* Gradients of sum(r . dr) + sum(a . da) (dr or da may be NULL: zeros): where
 * not NULL dx and dres per row (the same values, each in its type) and dweight,
 * dbias fp32 [channels] (summed over the rows in a fixed order; they need da).
 * The other arguments are those of the forward call that wrote `saved`.  dres may
 * be dr itself. */
fi_status fi_layer_backward(const fi_layer_desc *desc, const void *x, const void *res, const float *weight,
                            const float *saved, const void *dr, const void *da, void *dx, void *dres, float *dweight,
                            float *dbias, void *workspace, void *stream);

/* Matrix-vector products with 4-bit weights and group scales, for the block's
 * projections on the few rows of one position:
 *
 *     y[b][n] = sum_k x[b][k] scale[n][k / group] (code[n][k] - zero[n][k / group])
 *
 * codes 0..15; zero 0..15, or 8 everywhere where none are given.  The weights
 * are laid out once (fi_q4_pack) for the matrix instructions. */
typedef struct fi_q4_desc {
    int N, K;              /* outputs, inputs: 1 .. 2^20 each */
    int group;             /* 32, 64 or 128 values along K share a scale */
    int scale_dtype;       /* FI_F32, FI_BF16 or FI_F16 */
    int has_zeros;         /* 0: every zero is 8 */
    int reserved[3];       /* must be zero */
} fi_q4_desc;

/* Device bytes of the packed weights; 0 for a bad descriptor. */
size_t fi_q4_packed_bytes(const fi_q4_desc *desc);

/* codes [N][K] uint8 (the low four bits count), scales [N][ceil(K/group)] of
 * scale_dtype, zeros [N][ceil(K/group)] uint8 (NULL unless has_zeros), all
 * device memory, densely packed; packed 256-byte aligned. */
fi_status fi_q4_pack(const fi_q4_desc *desc, const uint8_t *codes, const void *scales, const uint8_t *zeros,
                     void *packed, void *stream);

/* Codes and scales of a weight matrix w [N][K] of w_dtype (row pitch ld_w
 * elements, 0 = K), zeros all 8: scale = max|w| of the group / 7 rounded to
 * scale_dtype, code = 8 + w / scale rounded to nearest even, in 1..15.  A
 * group of zeros, or one whose scale rounds to zero, gets scale 0 and codes 8.
 * w is finite, and max|w| / 7 in the range of scale_dtype. */
fi_status fi_q4_quantize(const fi_q4_desc *desc, int w_dtype, const void *w, int64_t ld_w, uint8_t *codes,
                         void *scales, void *stream);

/* y [rows][N] = x [rows][K] times the packed weights; rows 1 .. 16, x and y of
 * `dtype`.  fp32 inputs are multiplied in full (as three bf16 terms; below 2^-110
 * in size the last bits may be lost), 16-bit ones exactly too; sums are fp32.  A
 * row of x with an infinity or NaN gives non-finite values in its row of y only.
 * |x| stays below 2^116: then no sum within a group of 128 passes fp32's largest
 * number, whatever the codes and zeros ((32 x 31 + 96 x 15) 2^116 < 2^128). */
fi_status fi_q4_matvec(const fi_q4_desc *desc, const void *packed, int rows, int dtype, const void *x, int64_t ld_x,
                       void *y, int64_t ld_y, void *stream);

/* Products in 8-bit integers with a scale a row and a scale an output, for the
 * block's projections on any number of rows:
 *
 *     y[m][n] = sa[m] sw[n] sum_k a[m][k] w[n][k] + bias[n]
 *
 * Weights [N][K] and activations [rows][K] are kept alike: codes -128 .. 127 in
 * the order of the matrix instructions and an fp32 scale a row, laid out from
 * codes and scales (fi_q8_pack) or from values (fi_q8_quantize).  rows and N are
 * up to 2^24, K up to 131071 (the sums are whole numbers of 32 bits and exact),
 * rows * N up to 2^38. */

/* Device bytes of a packed matrix (256-byte aligned); 0 for a bad size. */
size_t fi_q8_bytes(int64_t rows, int K);

/* codes [rows][K] int8 and scales [rows] fp32, device memory, densely packed. */
fi_status fi_q8_pack(int64_t rows, int K, const int8_t *codes, const float *scales, void *packed, void *stream);

/* From values x [rows][K] of dtype (row pitch ld_x elements, 0 = K): scale =
 * max|x| of the row / 127 and code = x / scale rounded to nearest even, both
 * quotients in fp32.  A row whose scale rounds to zero gets codes 0; one with an
 * infinity or NaN gets a scale of NaN and gives NaN in its outputs only.  Below a
 * largest |x| of 2^-119 the scale is no normal number and has lost digits. */
fi_status fi_q8_quantize(int64_t rows, int K, int dtype, const void *x, int64_t ld_x, void *packed, void *stream);

/* y [rows][N] of dtype (row pitch ld_y elements, 0 = N); bias [N] fp32 or NULL.
 * The whole sum is rounded to fp32, multiplied by both scales and rounded once
 * more when it is stored. */
fi_status fi_q8_product(int64_t rows, int64_t N, int K, const void *a, const void *w, const float *bias, int dtype,
                        void *y, int64_t ld_y, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FI_H */
