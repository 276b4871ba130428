// Gated linear recurrence over packed sequences, its backward pass and its
// single-token form.
//
//   h_t = a_t h_{t-1} + u_t,   u_t = x_t, or (1 - a_t) x_t when coupled.
//
// The coupled form run back to front is the compositing recurrence
// S <- (1 - alpha) S + alpha c of "Gaussian Splatting反向传播的CUDA实现"
// (section 2) with gate 1 - alpha.  Its adjoint runs the other way:
//   g_t = dh_t + a_{t+1} g_{t+1},  da_t = g_t (h_{t-1} - [coupled] x_t),
//   dx_t = g_t (coupled: (1 - a_t) g_t).
//
// A run of rows acts on the state before it as h -> A h + B with A the
// product of its gates, and two runs compose as (A2 A1, A2 B1 + B2), so the
// time axis splits: thread runs inside a tile, tiles of a chunk of rows by a
// block of channels, and a chain of chunks joined by a decoupled look-back
// (a chunk publishes (A, B) as soon as it has it, and its state once the
// chunks before it are known).  One pass over HBM: a tile waits in shared
// memory while its carry is found.  A sequence's first row takes its state
// from h0, never from the row before it: a run that holds such a row absorbs
// (no 0 * inf between sequences), and so does its chunk, whose state is then
// published without looking back.
//
// Chunks are numbered by a ticket, so a chunk only ever waits for chunks
// that are already running; every wait is bounded.  States, products and
// gradients are fp32; each output is rounded once, when it is stored.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gs_internal.cuh"

namespace gs {
namespace {

constexpr int kScanBlock = 256;
// Rows per thread run.  Odd, so that the runs of one warp start in different
// banks for every power-of-two row size; at most 31 (start / finish bits of
// a run are one word).
constexpr int kRun = 17;
constexpr unsigned kSpinLimit = 1u << 20;

// How a tile moves between HBM and shared memory: 16-byte pieces of the
// whole tile (its rows are one contiguous range), 16-byte pieces of each
// row, or element by element.
enum CopyMode { kFlat = 0, kRow16 = 1, kElem = 2 };

struct ScanRecord {  // 16 bytes, published with one 128-bit store
    float A, B;
    unsigned tag;    // 2 * (epoch + 1) + (1 when B is the state after the chunk)
    unsigned pad;
};

struct ScanParams {
    long long rows, seq_len;
    const long long* offsets;  // NULL: n_seq sequences of seq_len rows
    long long sa, sx, sh, sda, sdx, sdh;
    int C, G, group;           // group = C / G channels per gate
    int n_seq, n_chunks, n_blocks;
    int lpr_log2;              // lanes per row, as a power of two
    int pitch, gate_pitch;     // elements of a tile row in shared memory
    int reverse, zero_pad, partial;
    int m_a, m_x, m_h, m_da, m_dx, m_dh;  // CopyMode
    const void *a, *x, *dh;
    const float *h0, *dh_last;
    void *h, *da, *dx;
    float *h_last, *states, *dh0, *part;
    WsHeader* hdr;
    ScanRecord* rec;
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int V> __device__ __forceinline__ void ld(const T* p, float (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = to_f<T>(p[0]);
    } else if constexpr (sizeof(T) == 4) {
        const float2 t = *reinterpret_cast<const float2*>(p);
        f[0] = t.x;
        f[1] = t.y;
    } else {
        const unsigned w = *reinterpret_cast<const unsigned*>(p);
        T e[2];
        memcpy(e, &w, 4);
        f[0] = to_f<T>(e[0]);
        f[1] = to_f<T>(e[1]);
    }
}

template <typename T, int V> __device__ __forceinline__ void st(T* p, const float (&f)[V]) {
    if constexpr (V == 1) {
        p[0] = from_f<T>(f[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
    } else {
        const T e[2] = {from_f<T>(f[0]), from_f<T>(f[1])};
        unsigned w;
        memcpy(&w, e, 4);
        *reinterpret_cast<unsigned*>(p) = w;
    }
}

// A h + B, where a zero state contributes nothing even if the product of the
// gates has overflowed (row by row, 0 * a is 0 for every finite gate; a gate
// that is not finite is in B already).
__device__ __forceinline__ float apply(float A, float B, float h) { return h == 0.0f ? B : fmaf(A, h, B); }

__device__ __forceinline__ void publish(ScanRecord* p, float A, float B, unsigned tag) {
    const unsigned long long lo = (unsigned long long)__float_as_uint(B) << 32 | __float_as_uint(A);
    const unsigned long long hi = tag;
    asm volatile("{ .reg .b128 q; mov.b128 q, {%1, %2}; st.relaxed.gpu.global.b128 [%0], q; }" ::"l"(p), "l"(lo),
                 "l"(hi)
                 : "memory");
}

__device__ __forceinline__ ScanRecord poll(const ScanRecord* p) {
    unsigned long long lo, hi;
    asm volatile("{ .reg .b128 q; ld.relaxed.gpu.global.b128 q, [%2]; mov.b128 {%0, %1}, q; }"
                 : "=l"(lo), "=l"(hi)
                 : "l"(p)
                 : "memory");
    ScanRecord r;
    r.A = __uint_as_float((unsigned)lo);
    r.B = __uint_as_float((unsigned)(lo >> 32));
    r.tag = (unsigned)hi;
    r.pad = 0;
    return r;
}

__device__ __forceinline__ void cp_async16(void* smem, const void* gmem) {
    const unsigned s = (unsigned)__cvta_generic_to_shared(smem);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Tile -> shared memory.  `cols` columns from `col0` of rows [r0, r0 + n);
// rows outside [lo, hi) (local) belong to no sequence and become `fill`.
template <typename T>
__device__ void load_tile(T* tile, const T* g, long long stride, long long r0, int n, int col0, int cols, int pitch,
                          int mode, int lo, int hi, float fill) {
    const int tid = threadIdx.x;
    constexpr int kPer = 16 / sizeof(T);
    if (lo == 0 && hi == n && mode != kElem) {
        if (mode == kFlat) {
            const int total = n * pitch, vecs = total / kPer;
            const T* src = g + r0 * stride;
            for (int i = tid; i < vecs; i += kScanBlock) cp_async16(tile + i * kPer, src + i * kPer);
            for (int i = vecs * kPer + tid; i < total; i += kScanBlock) tile[i] = src[i];
        } else {
            const int per = cols / kPer;
            for (int i = tid; i < n * per; i += kScanBlock) {
                const int r = i / per, v = i - r * per;
                cp_async16(tile + r * pitch + v * kPer, g + (r0 + r) * stride + col0 + v * kPer);
            }
        }
        return;
    }
    for (int i = tid; i < n * cols; i += kScanBlock) {
        const int r = i / cols, c = i - r * cols;
        tile[r * pitch + c] = (r >= lo && r < hi) ? g[(r0 + r) * stride + col0 + c] : from_f<T>(fill);
    }
}

// Shared memory -> tile; rows of no sequence are left as they were, or
// zeroed.
template <typename T>
__device__ void store_tile(const T* tile, T* g, long long stride, long long r0, int n, int col0, int cols, int pitch,
                           int mode, int lo, int hi, int zero_pad) {
    const int tid = threadIdx.x;
    constexpr int kPer = 16 / sizeof(T);
    if (lo == 0 && hi == n && mode != kElem) {
        if (mode == kFlat) {
            const int total = n * pitch, vecs = total / kPer;
            T* dst = g + r0 * stride;
            for (int i = tid; i < vecs; i += kScanBlock)
                reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(tile)[i];
            for (int i = vecs * kPer + tid; i < total; i += kScanBlock) dst[i] = tile[i];
        } else {
            const int per = cols / kPer;
            for (int i = tid; i < n * per; i += kScanBlock) {
                const int r = i / per, v = i - r * per;
                *reinterpret_cast<uint4*>(g + (r0 + r) * stride + col0 + v * kPer) =
                    *reinterpret_cast<const uint4*>(tile + r * pitch + v * kPer);
            }
        }
        return;
    }
    for (int i = tid; i < n * cols; i += kScanBlock) {
        const int r = i / cols, c = i - r * cols;
        const bool in = r >= lo && r < hi;
        if (in || zero_pad) g[(r0 + r) * stride + col0 + c] = in ? tile[r * pitch + c] : from_f<T>(0.0f);
    }
}

// Row offset of sequence j (j = n_seq: the end), clamped to the tensor so
// that bad offsets can give wrong values but no access out of range.
__device__ __forceinline__ long long seq_row(const ScanParams& p, long long j) {
    if (!p.offsets) return j * p.seq_len;
    const long long v = p.offsets[j];
    return v < 0 ? 0 : (v > p.rows ? p.rows : v);
}

// Smallest j in [0, n_seq + 1] with seq_row(j) >= row: a search with one
// probe per thread and round.
__device__ long long first_seq(const ScanParams& p, long long row) {
    if (!p.offsets) return p.seq_len > 0 ? (row + p.seq_len - 1) / p.seq_len : 0;
    long long lo = 0, n = (long long)p.n_seq + 1;
    while (n > 0) {
        const long long step = (n + kScanBlock - 1) / kScanBlock;
        const long long j = lo + (long long)threadIdx.x * step;
        const int below = __syncthreads_count(j < lo + n && seq_row(p, j) < row);
        // probes are increasing: the first `below` of them are below row
        if (below == 0) break;
        const long long nlo = lo + (long long)(below - 1) * step + 1;
        n = min(step - 1, lo + n - nlo);
        lo = nlo;
    }
    return lo;
}

// What the tile's rows are: per run the bits of rows that start (in scan
// order) or finish a sequence, and per row the sequence.
struct Marks {
    unsigned* start;   // [runs]
    unsigned* finish;  // [runs]
    int* start_seq;    // [tile rows], valid where the bit is set
    int* finish_seq;
};

// Fills the marks of rows [r0, r0 + n) of a tile of `bt` rows.  Sequences
// without rows pass their first state on: `from` -> `to` for the tile's
// channels (every such sequence belongs to exactly one chunk).
__device__ void mark_rows(const ScanParams& p, const Marks& mk, long long r0, int n, int bt, bool last_chunk,
                          const float* from, float* to, int c0, int nc) {
    const long long end = r0 + bt;
    for (long long j = first_seq(p, r0) + threadIdx.x; j <= p.n_seq; j += kScanBlock) {
        const long long v = seq_row(p, j);
        if (v > end) break;
        if (j < p.n_seq && (v < end || last_chunk)) {
            if (seq_row(p, j + 1) > v) {
                if (v < r0 + n && v >= r0) {
                    const int pr = (int)(v - r0);
                    const int l = p.reverse ? bt - 1 - pr : pr;
                    unsigned* bits = p.reverse ? mk.finish : mk.start;
                    (p.reverse ? mk.finish_seq : mk.start_seq)[pr] = (int)j;
                    atomicOr(&bits[l / kRun], 1u << (l % kRun));
                }
            } else if (to) {
                for (int c = 0; c < nc; ++c)
                    to[j * p.C + c0 + c] = from ? from[j * p.C + c0 + c] : 0.0f;
            }
        }
        if (j > 0 && v > r0 && v <= r0 + n && seq_row(p, j - 1) < v) {
            const int pr = (int)(v - 1 - r0);
            const int l = p.reverse ? bt - 1 - pr : pr;
            unsigned* bits = p.reverse ? mk.start : mk.finish;
            (p.reverse ? mk.start_seq : mk.finish_seq)[pr] = (int)(j - 1);
            atomicOr(&bits[l / kRun], 1u << (l % kRun));
        }
    }
}

// State of the scan in front of chunk k for every channel of the block, by
// looking back over the chunks before it (k > 0, none of this chunk's rows
// start a sequence or k's carry is needed for the rows before the first
// such row).  Threads (w, c) poll W chunks at a time; channel c's thread
// folds them from the nearest to the farthest.  False when a wait ran out.
__device__ bool look_back(const ScanParams& p, int k, int cb, int bc, unsigned tag, float* win, float* carry,
                          int* dead) {
    const int tid = threadIdx.x;
    int W = kScanBlock / bc;
    if (W > 32) W = 32;
    const int w = tid / bc, c = tid - w * bc;
    float Aacc = 1.0f, Bacc = 0.0f;
    bool done = false;
    for (int base = k - 1;; base -= W) {
        if (w < W) {
            const int idx = base - w;
            ScanRecord r;
            r.A = 0.0f;
            r.B = 0.0f;
            r.tag = tag + 1;
            if (idx >= 0) {
                const ScanRecord* q = p.rec + ((size_t)idx * p.n_blocks + cb) * bc + c;
                unsigned spin = 0;
                while (true) {
                    r = poll(q);
                    if ((r.tag | 1u) == (tag | 1u)) break;
                    if (++spin > kSpinLimit ||
                        ((spin & 1023u) == 0 && *reinterpret_cast<volatile unsigned*>(&p.hdr->status))) {
                        raise_status(p.hdr, GS_ERR_TIMEOUT);
                        *dead = 1;
                        r.A = r.B = 0.0f;
                        r.tag = tag + 1;
                        break;
                    }
                    __nanosleep(20);
                }
            }
            float* slot = win + (size_t)(w * bc + c) * 3;
            slot[0] = r.A;
            slot[1] = r.B;
            slot[2] = __uint_as_float(r.tag & 1u);
        }
        __syncthreads();
        if (tid < bc && !done) {
            for (int i = 0; i < W && !done; ++i) {
                const float* slot = win + (size_t)(i * bc + tid) * 3;
                Bacc = apply(Aacc, Bacc, slot[1]);
                if (__float_as_uint(slot[2])) done = true;
                else Aacc *= slot[0];
            }
        }
        if (__syncthreads_and(tid >= bc || done)) break;
    }
    if (tid < bc) carry[tid] = Bacc;
    __syncthreads();
    return *dead == 0;
}

// Shared memory of a tile kernel, carved from one dynamic block.
struct TileMem {
    char *x, *a, *g;
    Marks mk;
    float *wA, *wB, *carry, *win;
    int *flags, *wf;
};

__host__ __device__ inline size_t up16(size_t v) { return (v + 15) / 16 * 16; }

// Bytes of (and, on the device, pointers into) the dynamic shared memory.
__host__ __device__ inline size_t tile_mem(const ScanParams& p, int xs, int as, int v, bool bwd, char* base,
                                           TileMem* m) {
    const int lpr = 1 << p.lpr_log2, bc = lpr * v, runs = kScanBlock / lpr, bt = runs * kRun;
    const int warps = kScanBlock / 32;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        char* r = base + o;
        o += up16(bytes);
        return r;
    };
    char* x = take((size_t)bt * p.pitch * xs);
    char* a = take((size_t)bt * p.gate_pitch * as);
    char* g = bwd && p.dh ? take((size_t)bt * p.pitch * xs) : base;
    char* s0 = take((size_t)runs * 4);
    char* s1 = take((size_t)runs * 4);
    char* s2 = take((size_t)bt * 4);
    char* s3 = take((size_t)bt * 4);
    char* wa = take((size_t)warps * bc * 4);
    char* wb = take((size_t)warps * bc * 4);
    char* ca = take((size_t)bc * 4);
    char* wi = take((size_t)(kScanBlock > bc ? kScanBlock : bc) * 12);
    char* fl = take(16);
    char* wf = take(warps * 4);
    if (m) {
        m->x = x;
        m->a = a;
        m->g = g;
        m->mk = {reinterpret_cast<unsigned*>(s0), reinterpret_cast<unsigned*>(s1), reinterpret_cast<int*>(s2),
                 reinterpret_cast<int*>(s3)};
        m->wA = reinterpret_cast<float*>(wa);
        m->wB = reinterpret_cast<float*>(wb);
        m->carry = reinterpret_cast<float*>(ca);
        m->win = reinterpret_cast<float*>(wi);
        m->flags = reinterpret_cast<int*>(fl);
        m->wf = reinterpret_cast<int*>(wf);
    }
    return o;
}

// Which tile this block works on, and where it lies.
struct Tile {
    int k;            // chunk in the order the carry travels
    int chunk;        // chunk in row order
    int cb, c0, nc;   // channel block
    int bt, n;        // rows of a full tile, rows of this one
    int lo, hi;       // local range of the rows that belong to sequences
    long long r0;
    unsigned tag;     // record tag of an aggregate in this call
};

__device__ __forceinline__ Tile begin_tile(const ScanParams& p, int bc, bool descending, int* flags) {
    Tile t;
    unsigned id = blockIdx.x, epoch = 0;
    if (p.n_chunks > 1) {
        if (threadIdx.x == 0) {
            flags[1] = (int)atomicAdd(&p.hdr->ticket, 1u);
            flags[2] = (int)*reinterpret_cast<volatile unsigned*>(&p.hdr->reserved[0]);
        }
        __syncthreads();
        id = (unsigned)flags[1];
        epoch = (unsigned)flags[2];
    }
    t.tag = 2u * (epoch + 1u);
    t.k = (int)(id / (unsigned)p.n_blocks);
    t.cb = (int)(id - (unsigned)t.k * (unsigned)p.n_blocks);
    t.chunk = descending ? p.n_chunks - 1 - t.k : t.k;
    t.bt = (kScanBlock >> p.lpr_log2) * kRun;
    t.c0 = t.cb * bc;
    t.nc = min(bc, p.C - t.c0);
    t.r0 = (long long)t.chunk * t.bt;
    t.n = (int)max(0ll, min((long long)t.bt, p.rows - t.r0));
    long long lo = 0, hi = t.n;
    if (p.offsets) {
        lo = min(max(seq_row(p, 0) - t.r0, 0ll), (long long)t.n);
        hi = min(max(seq_row(p, p.n_seq) - t.r0, lo), (long long)t.n);
    }
    t.lo = (int)lo;
    t.hi = (int)hi;
    return t;
}

// The call's last block leaves the workspace ready for the next call: a new
// epoch makes every record stale.
__device__ __forceinline__ void end_tile(const ScanParams& p) {
    if (p.n_chunks <= 1) return;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        const unsigned total = (unsigned)p.n_chunks * (unsigned)p.n_blocks;
        if (atomicAdd(&p.hdr->reserved[1], 1u) == total - 1) {
            p.hdr->ticket = 0;
            p.hdr->reserved[1] = 0;
            p.hdr->reserved[0] += 1;
        }
    }
}

template <typename XT, typename AT, int V, bool COUPLED>
__global__ void __launch_bounds__(kScanBlock) k_scan_fwd(const __grid_constant__ ScanParams p) {
    extern __shared__ __align__(16) char smem[];
    TileMem m;
    tile_mem(p, sizeof(XT), sizeof(AT), V, false, smem, &m);
    const int tid = threadIdx.x, lane32 = tid & 31, warp = tid >> 5;
    const int lpr = 1 << p.lpr_log2, bc = lpr * V, runs = kScanBlock / lpr;
    const int run = tid >> p.lpr_log2, lane = tid & (lpr - 1);
    const Tile t = begin_tile(p, bc, p.reverse, m.flags);
    XT* sx = reinterpret_cast<XT*>(m.x);
    AT* sa = reinterpret_cast<AT*>(m.a);

    load_tile(sx, static_cast<const XT*>(p.x), p.sx, t.r0, t.n, t.c0, t.nc, p.pitch, p.m_x, t.lo, t.hi, 0.0f);
    const int g0 = t.c0 / p.group, ng = (t.c0 + t.nc - 1) / p.group - g0 + 1;
    load_tile(sa, static_cast<const AT*>(p.a), p.sa, t.r0, t.n, g0, ng, p.gate_pitch, p.m_a, t.lo, t.hi, 1.0f);
    for (int i = tid; i < runs; i += kScanBlock) m.mk.start[i] = m.mk.finish[i] = 0;
    if (tid == 0) m.flags[0] = 0;
    __syncthreads();
    mark_rows(p, m.mk, t.r0, t.n, t.bt, t.chunk == p.n_chunks - 1, p.h0, p.h_last, t.c0, t.nc);
    cp_async_wait();
    __syncthreads();

    const int ch = lane * V;
    const bool active = ch < t.nc;
    const int gate = active ? (t.c0 + ch) / p.group - g0 : 0;
    const unsigned starts = m.mk.start[run], finishes = m.mk.finish[run];
    const int l0 = run * kRun;
    // rows of the run that exist, as a range of r
    const int step = p.reverse ? -1 : 1;
    const int pr0 = p.reverse ? t.bt - 1 - l0 : l0;
    const int ra = p.reverse ? max(0, pr0 - t.n + 1) : 0;
    const int rb = p.reverse ? kRun : min(kRun, t.n - l0);

    float A[V], B[V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f;
    auto row = [&](int r, float (&av)[V], float (&uv)[V]) {
        const int pr = pr0 + step * r;
        if (p.group == 1) {
            ld<AT, V>(sa + pr * p.gate_pitch + ch, av);
        } else {
            av[0] = to_f<AT>(sa[pr * p.gate_pitch + gate]);
            if (V == 2) av[V - 1] = av[0];
        }
        ld<XT, V>(sx + pr * p.pitch + ch, uv);
        if (COUPLED) {
#pragma unroll
            for (int v = 0; v < V; ++v) uv[v] *= 1.0f - av[v];
        }
    };
    auto first = [&](int r, int v) {
        return p.h0 ? p.h0[(size_t)m.mk.start_seq[pr0 + step * r] * p.C + t.c0 + ch + v] : 0.0f;
    };
    if (active) {
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
            if (r < ra || r >= rb) continue;
            float av[V], uv[V];
            row(r, av, uv);
            const bool s = (starts >> r) & 1u;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                B[v] = fmaf(av[v], s ? first(r, v) : B[v], uv[v]);
                A[v] *= av[v];
            }
        }
    }
    // join the runs: inside the warp, then over the warps
    int f = starts != 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        if (d < lpr) continue;
        const int fo = __shfl_up_sync(~0u, f, d);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float Ao = __shfl_up_sync(~0u, A[v], d), Bo = __shfl_up_sync(~0u, B[v], d);
            if (lane32 >= d && !f) {
                B[v] = apply(A[v], B[v], Bo);
                A[v] *= Ao;
            }
        }
        if (lane32 >= d) f |= fo;
    }
    if (lane32 >= 32 - lpr) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            m.wA[warp * bc + ch + v] = A[v];
            m.wB[warp * bc + ch + v] = B[v];
        }
        if (lane32 == 31) m.wf[warp] = f;
    }
    // what lies before this run inside the warp
    int fe = __shfl_up_sync(~0u, f, lpr & 31);
    float Ae[V], Be[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        Ae[v] = __shfl_up_sync(~0u, A[v], lpr & 31);
        Be[v] = __shfl_up_sync(~0u, B[v], lpr & 31);
        if (lane32 < lpr) Ae[v] = 1.0f, Be[v] = 0.0f;
    }
    if (lane32 < lpr) fe = 0;
    __syncthreads();
    bool alive = true;
    if (p.n_chunks > 1) {
        float At = 1.0f, Bt = 0.0f;
        int ft = 0;
        ScanRecord* mine = p.rec + ((size_t)t.k * p.n_blocks + t.cb) * bc + tid;
        if (tid < bc) {
            for (int w = 0; w < kScanBlock / 32; ++w) {
                if (m.wf[w]) Bt = m.wB[w * bc + tid], ft = 1;
                else Bt = apply(m.wA[w * bc + tid], m.wB[w * bc + tid], Bt), At *= m.wA[w * bc + tid];
            }
            publish(mine, At, Bt, t.tag | (ft || t.k == 0 ? 1u : 0u));
        }
        if (t.k > 0) {
            alive = look_back(p, t.k, t.cb, bc, t.tag, m.win, m.carry, m.flags);
            if (tid < bc && !ft && alive) publish(mine, 0.0f, apply(At, Bt, m.carry[tid]), t.tag | 1u);
        } else {
            if (tid < bc) m.carry[tid] = 0.0f;
            __syncthreads();
        }
    } else {
        if (tid < bc) m.carry[tid] = 0.0f;
        __syncthreads();
    }
    if (alive) {
        if (p.states && tid < t.nc) p.states[(size_t)t.chunk * p.C + t.c0 + tid] = m.carry[tid];
        if (active) {
            float h[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                h[v] = m.carry[ch + v];
                for (int w = 0; w < warp; ++w)
                    h[v] = m.wf[w] ? m.wB[w * bc + ch + v]
                                   : apply(m.wA[w * bc + ch + v], m.wB[w * bc + ch + v], h[v]);
                h[v] = fe ? Be[v] : apply(Ae[v], Be[v], h[v]);
            }
#pragma unroll
            for (int r = 0; r < kRun; ++r) {
                if (r < ra || r >= rb) continue;
                float av[V], uv[V];
                row(r, av, uv);
                const bool s = (starts >> r) & 1u;
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = fmaf(av[v], s ? first(r, v) : h[v], uv[v]);
                if (p.h) st<XT, V>(sx + (pr0 + step * r) * p.pitch + ch, h);
                if (p.h_last && ((finishes >> r) & 1u)) {
                    float* q = p.h_last + (size_t)m.mk.finish_seq[pr0 + step * r] * p.C + t.c0 + ch;
#pragma unroll
                    for (int v = 0; v < V; ++v) q[v] = h[v];
                }
            }
        }
        __syncthreads();
        if (p.h)
            store_tile(sx, static_cast<XT*>(p.h), p.sh, t.r0, t.n, t.c0, t.nc, p.pitch, p.m_h, t.lo, t.hi,
                       p.zero_pad);
    }
    end_tile(p);
}

template <typename XT, typename AT, int V, bool COUPLED>
__global__ void __launch_bounds__(kScanBlock) k_scan_bwd(const __grid_constant__ ScanParams p) {
    extern __shared__ __align__(16) char smem[];
    TileMem m;
    tile_mem(p, sizeof(XT), sizeof(AT), V, true, smem, &m);
    const int tid = threadIdx.x, lane32 = tid & 31, warp = tid >> 5;
    const int lpr = 1 << p.lpr_log2, bc = lpr * V, runs = kScanBlock / lpr;
    const int run = tid >> p.lpr_log2, lane = tid & (lpr - 1);
    const Tile t = begin_tile(p, bc, !p.reverse, m.flags);
    XT* sx = reinterpret_cast<XT*>(m.x);
    AT* sa = reinterpret_cast<AT*>(m.a);
    XT* sg = reinterpret_cast<XT*>(m.g);

    load_tile(sx, static_cast<const XT*>(p.x), p.sx, t.r0, t.n, t.c0, t.nc, p.pitch, p.m_x, t.lo, t.hi, 0.0f);
    const int g0 = t.c0 / p.group, ng = (t.c0 + t.nc - 1) / p.group - g0 + 1;
    load_tile(sa, static_cast<const AT*>(p.a), p.sa, t.r0, t.n, g0, ng, p.gate_pitch, p.m_a, t.lo, t.hi, 1.0f);
    if (p.dh)
        load_tile(sg, static_cast<const XT*>(p.dh), p.sdh, t.r0, t.n, t.c0, t.nc, p.pitch, p.m_dh, t.lo, t.hi, 0.0f);
    for (int i = tid; i < runs; i += kScanBlock) m.mk.start[i] = m.mk.finish[i] = 0;
    if (tid == 0) m.flags[0] = 0;
    __syncthreads();
    mark_rows(p, m.mk, t.r0, t.n, t.bt, t.chunk == p.n_chunks - 1, p.dh_last, p.dh0, t.c0, t.nc);
    cp_async_wait();
    __syncthreads();

    const int ch = lane * V;
    const bool active = ch < t.nc;
    const int gate = active ? (t.c0 + ch) / p.group - g0 : 0;
    const unsigned starts = m.mk.start[run], finishes = m.mk.finish[run];
    const int l0 = run * kRun;
    const int step = p.reverse ? -1 : 1;
    const int pr0 = p.reverse ? t.bt - 1 - l0 : l0;
    const int ra = p.reverse ? max(0, pr0 - t.n + 1) : 0;
    const int rb = p.reverse ? kRun : min(kRun, t.n - l0);

    auto gates = [&](int pr, float (&av)[V]) {
        if (p.group == 1) {
            ld<AT, V>(sa + pr * p.gate_pitch + ch, av);
        } else {
            av[0] = to_f<AT>(sa[pr * p.gate_pitch + gate]);
            if (V == 2) av[V - 1] = av[0];
        }
    };
    auto first = [&](int pr, int v) {
        return p.h0 ? p.h0[(size_t)m.mk.start_seq[pr] * p.C + t.c0 + ch + v] : 0.0f;
    };
    // gradient a row's state receives from outside the recurrence
    auto upstream = [&](int r, int pr, float (&dv)[V]) {
#pragma unroll
        for (int v = 0; v < V; ++v) dv[v] = 0.0f;
        if (p.dh) ld<XT, V>(sg + pr * p.pitch + ch, dv);
        if (p.dh_last && ((finishes >> r) & 1u)) {
            const float* q = p.dh_last + (size_t)m.mk.finish_seq[pr] * p.C + t.c0 + ch;
#pragma unroll
            for (int v = 0; v < V; ++v) dv[v] += q[v];
        }
    };
    float A[V], B[V], K[V];  // the run on the state (A, B), and on the adjoint (A, K)
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f, K[v] = 0.0f;
    if (active) {
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
            if (r < ra || r >= rb) continue;
            const int pr = pr0 + step * r;
            float av[V], xv[V];
            gates(pr, av);
            ld<XT, V>(sx + pr * p.pitch + ch, xv);
            const bool s = (starts >> r) & 1u;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float u = COUPLED ? xv[v] * (1.0f - av[v]) : xv[v];
                B[v] = fmaf(av[v], s ? first(pr, v) : B[v], u);
                A[v] *= av[v];
            }
        }
#pragma unroll
        for (int r = kRun - 1; r >= 0; --r) {
            if (r < ra || r >= rb) continue;
            const int pr = pr0 + step * r;
            float av[V], dv[V];
            gates(pr, av);
            upstream(r, pr, dv);
            const bool s = (starts >> r) & 1u;
#pragma unroll
            for (int v = 0; v < V; ++v) K[v] = s ? 0.0f : av[v] * (dv[v] + K[v]);
        }
    }
    // join the runs on the state, forwards: what lies before this run
    const int f0 = starts != 0;
    float Ai[V], Bi[V];
    int f = f0;
#pragma unroll
    for (int v = 0; v < V; ++v) Ai[v] = A[v], Bi[v] = B[v];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        if (d < lpr) continue;
        const int fo = __shfl_up_sync(~0u, f, d);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float Ao = __shfl_up_sync(~0u, Ai[v], d), Bo = __shfl_up_sync(~0u, Bi[v], d);
            if (lane32 >= d && !f) {
                Bi[v] = apply(Ai[v], Bi[v], Bo);
                Ai[v] *= Ao;
            }
        }
        if (lane32 >= d) f |= fo;
    }
    if (lane32 >= 32 - lpr) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            m.wA[warp * bc + ch + v] = Ai[v];
            m.wB[warp * bc + ch + v] = Bi[v];
        }
        if (lane32 == 31) m.wf[warp] = f;
    }
    int fe = __shfl_up_sync(~0u, f, lpr & 31);
    float Ae[V], Be[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        Ae[v] = __shfl_up_sync(~0u, Ai[v], lpr & 31);
        Be[v] = __shfl_up_sync(~0u, Bi[v], lpr & 31);
        if (lane32 < lpr) Ae[v] = 1.0f, Be[v] = 0.0f;
    }
    if (lane32 < lpr) fe = 0;
    __syncthreads();
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        h[v] = active ? p.states[(size_t)t.chunk * p.C + t.c0 + ch + v] : 0.0f;
        for (int w = 0; w < warp; ++w)
            h[v] = m.wf[w] ? m.wB[w * bc + ch + v] : apply(m.wA[w * bc + ch + v], m.wB[w * bc + ch + v], h[v]);
        h[v] = fe ? Be[v] : apply(Ae[v], Be[v], h[v]);
    }
    __syncthreads();
    // join the runs on the adjoint, backwards: what lies behind this run
    f = f0;
#pragma unroll
    for (int v = 0; v < V; ++v) Ai[v] = A[v], Bi[v] = K[v];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        if (d < lpr) continue;
        const int fo = __shfl_down_sync(~0u, f, d);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float Ao = __shfl_down_sync(~0u, Ai[v], d), Bo = __shfl_down_sync(~0u, Bi[v], d);
            if (lane32 + d < 32 && !f) {
                Bi[v] = apply(Ai[v], Bi[v], Bo);
                Ai[v] *= Ao;
            }
        }
        if (lane32 + d < 32) f |= fo;
    }
    if (lane32 < lpr) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            m.wA[warp * bc + ch + v] = Ai[v];
            m.wB[warp * bc + ch + v] = Bi[v];
        }
        if (lane32 == 0) m.wf[warp] = f;
    }
    fe = __shfl_down_sync(~0u, f, lpr & 31);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        Ae[v] = __shfl_down_sync(~0u, Ai[v], lpr & 31);
        Be[v] = __shfl_down_sync(~0u, Bi[v], lpr & 31);
        if (lane32 + lpr >= 32) Ae[v] = 1.0f, Be[v] = 0.0f;
    }
    if (lane32 + lpr >= 32) fe = 0;
    __syncthreads();
    bool alive = true;
    const int nw = kScanBlock / 32;
    if (p.n_chunks > 1) {
        float At = 1.0f, Bt = 0.0f;
        int ft = 0;
        ScanRecord* mine = p.rec + ((size_t)t.k * p.n_blocks + t.cb) * bc + tid;
        if (tid < bc) {
            for (int w = nw - 1; w >= 0; --w) {
                if (m.wf[w]) Bt = m.wB[w * bc + tid], ft = 1;
                else Bt = apply(m.wA[w * bc + tid], m.wB[w * bc + tid], Bt), At *= m.wA[w * bc + tid];
            }
            publish(mine, At, Bt, t.tag | (ft || t.k == 0 ? 1u : 0u));
        }
        if (t.k > 0) {
            alive = look_back(p, t.k, t.cb, bc, t.tag, m.win, m.carry, m.flags);
            if (tid < bc && !ft && alive) publish(mine, 0.0f, apply(At, Bt, m.carry[tid]), t.tag | 1u);
        } else {
            if (tid < bc) m.carry[tid] = 0.0f;
            __syncthreads();
        }
    } else {
        if (tid < bc) m.carry[tid] = 0.0f;
        __syncthreads();
    }
    if (alive) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float k = m.carry[ch + v];
            for (int w = nw - 1; w > warp; --w)
                k = m.wf[w] ? m.wB[w * bc + ch + v] : apply(m.wA[w * bc + ch + v], m.wB[w * bc + ch + v], k);
            K[v] = fe ? Be[v] : apply(Ae[v], Be[v], k);
        }
        float hp[kRun][V];  // state before each row
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
#pragma unroll
            for (int v = 0; v < V; ++v) hp[r][v] = 0.0f;
            if (r < ra || r >= rb || !active) continue;
            const int pr = pr0 + step * r;
            float av[V], xv[V];
            gates(pr, av);
            ld<XT, V>(sx + pr * p.pitch + ch, xv);
            const bool s = (starts >> r) & 1u;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float u = COUPLED ? xv[v] * (1.0f - av[v]) : xv[v];
                hp[r][v] = s ? first(pr, v) : h[v];
                h[v] = fmaf(av[v], hp[r][v], u);
            }
        }
        // lanes of the row that share this lane's gate, by distance
        unsigned same = 0;
        if (p.group > 1 && active) {
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const int o = lane + (1 << i);
                if (o < lpr && o * V < t.nc && (t.c0 + o * V) / p.group - g0 == gate) same |= 1u << i;
            }
        }
        const bool head = active && (ch == 0 || (t.c0 + ch - 1) / p.group - g0 != gate);
#pragma unroll
        for (int r = kRun - 1; r >= 0; --r) {
            const int pr = pr0 + step * r;
            const bool in = r >= ra && r < rb && active;
            float dav[V];
#pragma unroll
            for (int v = 0; v < V; ++v) dav[v] = 0.0f;
            if (in) {
                float av[V], dv[V], xv[V], dxv[V];
                gates(pr, av);
                upstream(r, pr, dv);
                if (COUPLED) ld<XT, V>(sx + pr * p.pitch + ch, xv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float g = dv[v] + K[v];
                    dav[v] = g * (COUPLED ? hp[r][v] - xv[v] : hp[r][v]);
                    dxv[v] = COUPLED ? g * (1.0f - av[v]) : g;
                    K[v] = av[v] * g;
                }
                if ((starts >> r) & 1u) {
                    if (p.dh0) {
                        float* q = p.dh0 + (size_t)m.mk.start_seq[pr] * p.C + t.c0 + ch;
#pragma unroll
                        for (int v = 0; v < V; ++v) q[v] = K[v];
                    }
#pragma unroll
                    for (int v = 0; v < V; ++v) K[v] = 0.0f;
                }
                st<XT, V>(sx + pr * p.pitch + ch, dxv);
            }
            if (p.group == 1) {
                if (in) st<AT, V>(sa + pr * p.gate_pitch + ch, dav);
            } else {
                float s = V == 2 ? dav[0] + dav[V - 1] : dav[0];
#pragma unroll
                for (int i = 0; i < 5; ++i) {
                    if ((1 << i) >= lpr) continue;
                    const float o = __shfl_down_sync(~0u, s, 1 << i);
                    if ((same >> i) & 1u) s += o;
                }
                if (in && head) {
                    if (p.partial)
                        p.part[((size_t)t.cb * p.rows + t.r0 + pr) * p.gate_pitch + gate] = s;
                    else
                        sa[pr * p.gate_pitch + gate] = from_f<AT>(s);
                }
            }
        }
        __syncthreads();
        store_tile(sx, static_cast<XT*>(p.dx), p.sdx, t.r0, t.n, t.c0, t.nc, p.pitch, p.m_dx, t.lo, t.hi, p.zero_pad);
        if (!p.partial)
            store_tile(sa, static_cast<AT*>(p.da), p.sda, t.r0, t.n, g0, ng, p.gate_pitch, p.m_da, t.lo, t.hi,
                       p.zero_pad);
    }
    end_tile(p);
}

// Gate gradients of groups that lie in several channel blocks: the blocks'
// parts, added in order.
template <typename AT>
__global__ void __launch_bounds__(kScanBlock) k_gate_sum(const __grid_constant__ ScanParams p, int bc) {
    const long long total = p.rows * p.G;
    long long lo = 0, hi = p.rows;
    if (p.offsets) lo = seq_row(p, 0), hi = seq_row(p, p.n_seq);
    for (long long i = (long long)blockIdx.x * kScanBlock + threadIdx.x; i < total;
         i += (long long)gridDim.x * kScanBlock) {
        const long long r = i / p.G;
        const int g = (int)(i - r * p.G);
        AT* out = static_cast<AT*>(p.da) + r * p.sda + g;
        if (r < lo || r >= hi) {
            if (p.zero_pad) *out = from_f<AT>(0.0f);
            continue;
        }
        const int c0 = g * p.group, b0 = c0 / bc, b1 = (c0 + p.group - 1) / bc;
        float s = 0.0f;
        for (int b = b0; b <= b1; ++b)
            s += p.part[((size_t)b * p.rows + r) * p.gate_pitch + g - b * bc / p.group];
        *out = from_f<AT>(s);
    }
}

// One row of the recurrence for every kept state: elementwise.
template <typename XT, typename AT, int V>
__global__ void __launch_bounds__(kScanBlock)
k_scan_step(long long n, int C, int G, int group, int coupled, long long sa, long long sx, long long sh, const AT* a,
            const XT* x, const float* state, float* state_out, XT* h) {
    const int per = C / V;
    for (long long i = (long long)blockIdx.x * kScanBlock + threadIdx.x; i < n * per;
         i += (long long)gridDim.x * kScanBlock) {
        const long long r = i / per;
        const int c = (int)(i - r * per) * V;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float av = to_f<AT>(a[r * sa + (group == 1 ? c + v : (c + v) / group)]);
            float u = to_f<XT>(x[r * sx + c + v]);
            if (coupled) u *= 1.0f - av;
            const float s = fmaf(av, state[r * C + c + v], u);
            state_out[r * C + c + v] = s;
            if (h) h[r * sh + c + v] = from_f<XT>(s);
        }
    }
}

// ---- host ---------------------------------------------------------------

int elem_size(int dtype) { return dtype == GS_F32 ? 4 : 2; }

struct Plan {
    ScanParams p;
    int v, bc, bt;
    size_t rec_bytes, part_bytes;
};

// Checks the description and chooses the tiling.
bool make_plan(const gs_scan_desc* d, Plan* out) {
    if (!d) return false;
    if (d->rows < 0 || d->n_seq < 0 || d->channels < 1 || d->gates < 1 || d->channels % d->gates) return false;
    if (d->dtype != GS_F32 && d->dtype != GS_BF16 && d->dtype != GS_F16) return false;
    if (d->gate_dtype != GS_F32 && d->gate_dtype != d->dtype) return false;
    if (d->flags & ~(GS_SCAN_REVERSE | GS_SCAN_COUPLED | GS_SCAN_ZERO_PAD)) return false;
    const long long C = d->channels, G = d->gates, lim = 1ll << 40;
    for (long long s : {d->stride_x, d->stride_h, d->stride_dh, d->stride_dx})
        if (s < C || s > lim) return false;
    for (long long s : {d->stride_a, d->stride_da})
        if (s < G || s > lim) return false;
    if (d->rows > lim || (d->rows > 0 && d->n_seq == 0)) return false;
    Plan& q = *out;
    q.p = ScanParams{};
    ScanParams& p = q.p;
    p.rows = d->rows;
    p.n_seq = d->n_seq;
    p.C = d->channels;
    p.G = d->gates;
    p.group = p.C / p.G;
    p.sa = d->stride_a, p.sx = d->stride_x, p.sh = d->stride_h;
    p.sda = d->stride_da, p.sdx = d->stride_dx, p.sdh = d->stride_dh;
    p.reverse = (d->flags & GS_SCAN_REVERSE) != 0;
    p.zero_pad = (d->flags & GS_SCAN_ZERO_PAD) != 0;
    // 16-bit channels go two to a thread where pairs share their gate or have one each
    q.v = d->dtype != GS_F32 && p.C % 2 == 0 && (p.group == 1 || p.group % 2 == 0) ? 2 : 1;
    const int lanes = (p.C + q.v - 1) / q.v;
    while ((1 << p.lpr_log2) < lanes && p.lpr_log2 < 5) ++p.lpr_log2;
    const int lpr = 1 << p.lpr_log2;
    q.bc = lpr * q.v;
    q.bt = kScanBlock / lpr * kRun;
    p.n_blocks = (p.C + q.bc - 1) / q.bc;
    p.pitch = p.n_blocks > 1 ? q.bc : p.C;
    const long long chunks = d->rows > 0 ? (d->rows + q.bt - 1) / q.bt : 1;
    if (chunks * p.n_blocks > 0x7fffffffll) return false;
    p.n_chunks = (int)chunks;
    if (p.group == 1) {
        p.gate_pitch = p.pitch;
    } else if (p.n_blocks == 1) {
        p.gate_pitch = p.G;
    } else {
        p.gate_pitch = q.bc % p.group == 0 ? q.bc / p.group : (p.group % q.bc == 0 ? 1 : (q.bc - 1) / p.group + 2);
        if (p.gate_pitch > p.G) p.gate_pitch = p.G;
    }
    p.partial = p.n_blocks > 1 && p.group > 1 && q.bc % p.group != 0;
    q.rec_bytes = p.n_chunks > 1 ? (size_t)p.n_chunks * p.n_blocks * q.bc * sizeof(ScanRecord) : 0;
    q.part_bytes = p.partial ? align_up((size_t)p.n_blocks * p.rows * p.gate_pitch * 4, 16) : 0;
    return true;
}

size_t plan_ws(const Plan& q) {
    return q.rec_bytes + q.part_bytes ? sizeof(WsHeader) + q.rec_bytes + q.part_bytes : 0;
}

int copy_mode(const Plan& q, const void* ptr, long long stride, int es, int cols, int pitch, bool gate) {
    const ScanParams& p = q.p;
    if (!aligned(ptr, 16)) return kElem;
    // whole rows, one after another, and the same columns for every block
    if (pitch == cols && stride == cols && (p.n_blocks == 1 || cols == 1)) return kFlat;
    if (gate && p.group > 1) return kElem;
    if (stride * es % 16 == 0 && cols * es % 16 == 0 && pitch * es % 16 == 0) return kRow16;
    return kElem;
}

void set_workspace(Plan& q, void* ws) {
    q.p.hdr = static_cast<WsHeader*>(ws);
    char* b = static_cast<char*>(ws) + sizeof(WsHeader);
    q.p.rec = reinterpret_cast<ScanRecord*>(b);
    q.p.part = reinterpret_cast<float*>(b + q.rec_bytes);
}

template <typename XT, typename AT, int V>
int launch_tiles(Plan& q, bool coupled, bool bwd, cudaStream_t s) {
    const size_t smem = tile_mem(q.p, sizeof(XT), sizeof(AT), V, bwd, nullptr, nullptr);
    const unsigned grid = (unsigned)(q.p.n_chunks) * (unsigned)q.p.n_blocks;
    auto k = bwd ? (coupled ? k_scan_bwd<XT, AT, V, true> : k_scan_bwd<XT, AT, V, false>)
                 : (coupled ? k_scan_fwd<XT, AT, V, true> : k_scan_fwd<XT, AT, V, false>);
    opt_in_smem(k, 227 * 1024);
    k<<<grid, kScanBlock, smem, s>>>(q.p); note_launch();
    GS_LAUNCH_CHECK();
    if (bwd && q.p.partial && q.p.rows > 0) {
        long long blocks = (q.p.rows * q.p.G + kScanBlock - 1) / kScanBlock;
        if (blocks > 148 * 8) blocks = 148 * 8;
        k_gate_sum<AT><<<(unsigned)blocks, kScanBlock, 0, s>>>(q.p, q.bc); note_launch();
        GS_LAUNCH_CHECK();
    }
    return GS_OK;
}

template <typename XT, typename AT>
int launch_v(Plan& q, bool coupled, bool bwd, cudaStream_t s) {
    if constexpr (sizeof(XT) == 2) {
        if (q.v == 2) return launch_tiles<XT, AT, 2>(q, coupled, bwd, s);
    }
    return launch_tiles<XT, AT, 1>(q, coupled, bwd, s);
}

int launch_typed(Plan& q, const gs_scan_desc* d, bool bwd, cudaStream_t s) {
    const bool c = (d->flags & GS_SCAN_COUPLED) != 0;
    if (d->dtype == GS_F32) return launch_v<float, float>(q, c, bwd, s);
    if (d->dtype == GS_BF16)
        return d->gate_dtype == GS_F32 ? launch_v<__nv_bfloat16, float>(q, c, bwd, s)
                                       : launch_v<__nv_bfloat16, __nv_bfloat16>(q, c, bwd, s);
    return d->gate_dtype == GS_F32 ? launch_v<__half, float>(q, c, bwd, s) : launch_v<__half, __half>(q, c, bwd, s);
}

bool set_sequences(Plan& q, const long long* offsets) {
    q.p.offsets = offsets;
    if (offsets) return aligned(offsets, 8);
    if (q.p.rows % (q.p.n_seq > 0 ? q.p.n_seq : 1)) return false;
    q.p.seq_len = q.p.n_seq > 0 ? q.p.rows / q.p.n_seq : 0;
    return true;
}

template <typename XT, typename AT>
int launch_step(const gs_scan_desc* d, const void* a, const void* x, const float* state, float* state_out, void* h,
                cudaStream_t s) {
    const long long n = d->rows * d->channels;
    long long blocks = (n + kScanBlock - 1) / kScanBlock;
    if (blocks > 148 * 8) blocks = 148 * 8;
    k_scan_step<XT, AT, 1><<<(unsigned)blocks, kScanBlock, 0, s>>>(
        d->rows, d->channels, d->gates, d->channels / d->gates, (d->flags & GS_SCAN_COUPLED) != 0, d->stride_a,
        d->stride_x, d->stride_h, static_cast<const AT*>(a), static_cast<const XT*>(x), state, state_out,
        static_cast<XT*>(h)); note_launch();
    GS_LAUNCH_CHECK();
    return GS_OK;
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" size_t gs_scan_workspace_bytes(const gs_scan_desc* desc) {
    Plan q;
    return make_plan(desc, &q) ? plan_ws(q) : 0;
}

extern "C" size_t gs_scan_states_bytes(const gs_scan_desc* desc) {
    Plan q;
    return make_plan(desc, &q) ? (size_t)q.p.n_chunks * q.p.C * sizeof(float) : 0;
}

extern "C" int gs_scan_fwd(const gs_scan_desc* desc, const void* a, const void* x, const float* h0,
                           const long long* seq_offsets, void* h, float* h_last, float* states, void* ws,
                           size_t ws_bytes, void* stream) {
    Plan q;
    if (!make_plan(desc, &q) || !set_sequences(q, seq_offsets)) return GS_ERR_INVALID_ARG;
    if (desc->n_seq == 0) return GS_OK;
    const int xs = elem_size(desc->dtype), as = elem_size(desc->gate_dtype);
    if (desc->rows > 0 && (!a || !x || !aligned(a, as) || !aligned(x, xs))) return GS_ERR_INVALID_ARG;
    if (!h && !h_last) return GS_ERR_INVALID_ARG;
    if (!aligned(h, xs) || !aligned(h0, 4) || !aligned(h_last, 4) || !aligned(states, 4)) return GS_ERR_INVALID_ARG;
    const size_t need = plan_ws(q);
    if (need && (!ws || ws_bytes < need || !aligned(ws, 16))) return GS_ERR_INVALID_ARG;
    ScanParams& p = q.p;
    p.a = a, p.x = x, p.h0 = h0, p.h = h, p.h_last = h_last, p.states = states;
    p.m_a = copy_mode(q, a, p.sa, as, p.G, p.gate_pitch, true);
    p.m_x = copy_mode(q, x, p.sx, xs, p.C, p.pitch, false);
    p.m_h = copy_mode(q, h, p.sh, xs, p.C, p.pitch, false);
    if (need) set_workspace(q, ws);
    return launch_typed(q, desc, false, (cudaStream_t)stream);
}

extern "C" int gs_scan_bwd(const gs_scan_desc* desc, const void* a, const void* x, const float* h0,
                           const long long* seq_offsets, const float* states, const void* dL_dh,
                           const float* dL_dh_last, void* dL_da, void* dL_dx, float* dL_dh0, void* ws,
                           size_t ws_bytes, void* stream) {
    Plan q;
    if (!make_plan(desc, &q) || !set_sequences(q, seq_offsets)) return GS_ERR_INVALID_ARG;
    if (desc->n_seq == 0) return GS_OK;
    const int xs = elem_size(desc->dtype), as = elem_size(desc->gate_dtype);
    if (desc->rows > 0 && (!a || !x || !dL_da || !dL_dx || !states || !aligned(a, as) || !aligned(x, xs) ||
                           !aligned(dL_da, as) || !aligned(dL_dx, xs)))
        return GS_ERR_INVALID_ARG;
    if (!aligned(dL_dh, xs) || !aligned(h0, 4) || !aligned(dL_dh_last, 4) || !aligned(dL_dh0, 4) ||
        !aligned(states, 4))
        return GS_ERR_INVALID_ARG;
    const size_t need = plan_ws(q);
    if (need && (!ws || ws_bytes < need || !aligned(ws, 16))) return GS_ERR_INVALID_ARG;
    if (desc->rows == 0 && !dL_dh0) return GS_OK;
    ScanParams& p = q.p;
    p.a = a, p.x = x, p.h0 = h0, p.states = const_cast<float*>(states);
    p.dh = dL_dh, p.dh_last = dL_dh_last, p.da = dL_da, p.dx = dL_dx, p.dh0 = dL_dh0;
    p.m_a = copy_mode(q, a, p.sa, as, p.G, p.gate_pitch, true);
    p.m_x = copy_mode(q, x, p.sx, xs, p.C, p.pitch, false);
    p.m_dh = copy_mode(q, dL_dh, p.sdh, xs, p.C, p.pitch, false);
    p.m_da = copy_mode(q, dL_da, p.sda, as, p.G, p.gate_pitch, true);
    p.m_dx = copy_mode(q, dL_dx, p.sdx, xs, p.C, p.pitch, false);
    if (need) set_workspace(q, ws);
    return launch_typed(q, desc, true, (cudaStream_t)stream);
}

extern "C" int gs_scan_step(const gs_scan_desc* desc, const void* a, const void* x, const float* state,
                            float* state_out, void* h, void* stream) {
    Plan q;
    if (!make_plan(desc, &q) || desc->n_seq != desc->rows) return GS_ERR_INVALID_ARG;
    if (desc->rows == 0) return GS_OK;
    const int xs = elem_size(desc->dtype), as = elem_size(desc->gate_dtype);
    if (!a || !x || !state || !state_out || !aligned(a, as) || !aligned(x, xs) || !aligned(state, 4) ||
        !aligned(state_out, 4) || !aligned(h, xs))
        return GS_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (desc->dtype == GS_F32) return launch_step<float, float>(desc, a, x, state, state_out, h, s);
    if (desc->dtype == GS_BF16)
        return desc->gate_dtype == GS_F32
                   ? launch_step<__nv_bfloat16, float>(desc, a, x, state, state_out, h, s)
                   : launch_step<__nv_bfloat16, __nv_bfloat16>(desc, a, x, state, state_out, h, s);
    return desc->gate_dtype == GS_F32 ? launch_step<__half, float>(desc, a, x, state, state_out, h, s)
                                      : launch_step<__half, __half>(desc, a, x, state, state_out, h, s);
}
