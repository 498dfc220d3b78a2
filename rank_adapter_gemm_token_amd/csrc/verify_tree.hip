// verify_tree.hip -- drafted trees walked down along the tokens drawn from the
// target's probabilities, from given random numbers.
//
// At a node with the weights w = max(0, p) of its row and the number u, the
// token is the first index at which the running sum of w, in fp64, passes u
// times the whole; the walk goes on at the first child that holds it.
//
// A row is cut into 64 chunks of neighbouring segments of 512 entries.  Its
// chunks are added up by the waves, each on its own; the chunk, the segment in
// it, the lane and the entry are then found by running sums of the wave's
// lanes.  Only the chunk that is drawn from is read again (a few KB).
//
// Bound by latency for one tree (32 nodes of 32000 entries, fp32: 9 us).  Where
// every row is drawn from at once (64 trees of up to 16, 131072 entries of 16
// bits: 142 MB in 40 us, 3.6 TB/s, of 6.7 that reads alone reach), by reads and
// draws that do not overlap: all workgroups run at once, read together, and then
// go through the draws' barriers and second reads together.
#include "dtype.hpp"
#include "kv_internal.hpp"
#include "row_eight.hpp"
#include "wave_fp64.hpp"

namespace lora {

namespace {

constexpr int STEP = 8;           // neighbouring entries of a lane
constexpr int SEGMENT = 64 * STEP;
constexpr int CHUNKS = VERIFY_CHUNKS;
constexpr int AHEAD = 4;          // segments a wave asks for together (8: a walk over 131072 entries 92 us instead of 89)
static_assert(CHUNKS == 64, "a lane for each");

// Entries i .. i + 7 of a row of V as weights: what is not above zero (NaN, what
// is past the end) counts as nothing.
template <int DT>
struct Weights {
    Eight<DT> e;
    __device__ __forceinline__ void load(const typename Elem<DT>::raw *row, int i, int V) { e.load(row, i, V); }
    // After load(); `whole`: no lane of the wave looks past the end.
    __device__ __forceinline__ void clear(int i, int V, bool whole) {
        if (!whole) e.clear(i, V, 0);
    }
    __device__ __forceinline__ double at(int j) const { return static_cast<double>(fmaxf(e.at(j), 0.0f)); }
    __device__ __forceinline__ double sum() const {
        double v = 0.0;
#pragma unroll
        for (int j = 0; j < STEP; ++j) v += at(j);
        return v;
    }
};

// What a workgroup of N threads needs to draw from a row.
struct Drawing {
    double chunk[CHUNKS];
    double segment[VERIFY_MAX_SEGMENTS];  // of the chunk drawn from
    int token;
};

template <int DT, int N>
struct Row {
    using raw = typename Elem<DT>::raw;
    static constexpr int WAVES = N / 64;
    const raw *p;
    int V, segments;  // of a chunk
    Drawing &sh;

    // Sums of chunks c0 .. c1 - 1, each by one wave.
    __device__ __forceinline__ void add(int c0, int c1) const {
        const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
        // None of a chunk past the row's end.
        if (threadIdx.x < CHUNKS) sh.chunk[threadIdx.x] = 0.0;
        __syncthreads();
        const int some = (V + segments * SEGMENT - 1) / (segments * SEGMENT);
        c1 = c1 < some ? c1 : some;
        int c = c0 + wave, s = 0;  // the next segment
        double acc = 0.0;
        while (c < c1) {
            Weights<DT> w[AHEAD];
            int cc = c, ss = s, at[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                at[k] = cc < c1 ? (cc * segments + ss) * SEGMENT : V;
                w[k].load(p, at[k] + lane * STEP, V);
                if (++ss == segments) ss = 0, cc += WAVES;
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (c >= c1) break;
                w[k].clear(at[k] + lane * STEP, V, at[k] + SEGMENT <= V);
                acc += w[k].sum();
                if (++s == segments) {
                    const double all = wave_sum(acc);
                    if (lane == 0) sh.chunk[c] = all;
                    acc = 0.0;
                    s = 0;
                    c += WAVES;
                }
            }
        }
    }

    // The token at which the running sum passes u times the whole, to all
    // threads; -1: the row has no weight, or no finite sum.  v: lane i has chunk
    // i's sum, in every wave.
    __device__ __forceinline__ int pick(double v, double u) const {
        const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
        double run = wave_scan(v);
        const double total = lane_of(run, 63), aim = u * total;
        if (!(total > 0.0 && total <= 1.7976931348623157e308)) return -1;
        const int c = pick_lane(v, run, aim);
        double base = c > 0 ? lane_of(run, c - 1) : 0.0;
        int s = 0;
        if (segments > 1) {
            for (int i = wave; i < segments; i += WAVES) {
                const int at = (c * segments + i) * SEGMENT;
                Weights<DT> w;
                w.load(p, at + lane * STEP, V);
                w.clear(at + lane * STEP, V, at + SEGMENT <= V);
                const double all = wave_sum(w.sum());
                if (lane == 0) sh.segment[i] = all;
            }
            __syncthreads();
            v = lane < segments ? sh.segment[lane] : 0.0;
            run = base + wave_scan(v);
            s = pick_lane(v, run, aim);
            if (s > 0) base = lane_of(run, s - 1);
        }
        if (wave == 0) {
            const int i = (c * segments + s) * SEGMENT + lane * STEP, first = V < STEP ? 0 : Eight<DT>::first(i, V);
            Weights<DT> w;
            w.load(p, i, V);
            w.clear(i, V, false);
            const double mine = w.sum(), upto = base + wave_scan(mine);
            const int l = pick_lane(mine, upto, aim);
            if (l > 0) base = lane_of(upto, l - 1);
            if (lane == l) {
                int hit = -1, last = -1;
#pragma unroll
                for (int j = 0; j < STEP; ++j) {
                    const double x = w.at(j);
                    base += x;
                    if (x > 0.0) last = first + j;
                    if (hit < 0 && x > 0.0 && base > aim) hit = first + j;
                }
                sh.token = hit >= 0 ? hit : last;  // last: rounding kept the sum at or below the aim
            }
        }
        __syncthreads();
        return sh.token;
    }
};

// Whether sequence b's rows r0 .. r1 - 1 leave at least one for each sequence
// before and after it.  (The bounds are compared before their difference is
// made, which may pass 32 bits.)
__device__ __forceinline__ bool rows_fit(const VerifyTreeArgs &a, int b, int r0, int r1) {
    return r0 >= b && r1 > r0 && r1 <= a.n_rows - (a.n_seqs - 1 - b);
}

// Workgroup b walks down sequence b's tree.  No row is read that the walk does
// not come by, but a row's draw waits for the one above it.
template <int DT, int N>
__global__ __launch_bounds__(N) void k_verify_walk(VerifyTreeArgs a) {
    const int b = blockIdx.x, t = threadIdx.x, lane = t & 63;
    __shared__ Drawing sh;
    __shared__ int child;
    const int r0 = a.row0[b], r1 = a.row0[b + 1];
    if (!rows_fit(a, b, r0, r1)) {
        if (t == 0) a.accepted[b] = -1;
        return;
    }
    const int n = r1 - r0;
    const int32_t *parent = a.parent + r0, *draft = a.draft + r0;
    // The first N nodes, a thread each.
    const int my_parent = t < n ? parent[t] : -1, my_draft = t < n ? draft[t] : -1;
    int node = 0, kept = 0;
    for (;;) {
        const Row<DT, N> row{static_cast<const typename Elem<DT>::raw *>(a.p) + static_cast<long>(r0 + node) * a.vocab,
                             a.vocab, a.segments, sh};
        const double u = static_cast<double>(a.u[r0 + node]);
        if (t == 0) child = n;
        row.add(0, CHUNKS);
        __syncthreads();
        const int token = row.pick(sh.chunk[lane], u);
        if (token < 0) {
            kept = -1;
            break;
        }
        if (t == 0) {
            a.tokens[r0 + kept] = token;
            a.path[r0 + kept] = node;
        }
        // A child comes after its parent, so the walk ends.
        if (t > node && t < n && my_parent == node && my_draft == token) atomicMin(&child, t);
        for (int j = t + N; j < n; j += N)
            if (j > node && parent[j] == node && draft[j] == token) atomicMin(&child, j);
        __syncthreads();
        const int next = child;
        __syncthreads();
        if (next >= n) break;
        node = next;
        ++kept;
    }
    if (t == 0) a.accepted[b] = kept;
    __syncthreads();
    for (int j = kept + 1 + t; j < n; j += N) a.tokens[r0 + j] = a.path[r0 + j] = -1;
}

__device__ __forceinline__ int get(const int *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Workgroup (r, c) adds up `group` of row r's chunks, the last of a row's
// workgroups draws its token, and the last of a sequence's rows walks down the
// tree along the tokens, which wait for it in the output.
template <int DT, int N>
__global__ __launch_bounds__(N) void k_verify_rows(VerifyTreeArgs a) {
    constexpr int NODES = 512;  // of a tree that is walked in LDS
    const int r = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6);
    __shared__ Drawing sh;
    __shared__ int seq, steps, lds[2 * NODES];
    __shared__ unsigned arrived;
    if (blockIdx.y == 0 && t == 0 && r < a.n_seqs && !rows_fit(a, r, a.row0[r], a.row0[r + 1])) a.accepted[r] = -1;
    if (r >= a.n_rows) return;

    const Row<DT, N> row{static_cast<const typename Elem<DT>::raw *>(a.p) + static_cast<long>(r) * a.vocab, a.vocab,
                         a.segments, sh};
    const double u = static_cast<double>(a.u[r]);
    const int c0 = blockIdx.y * a.group, c1 = c0 + a.group < CHUNKS ? c0 + a.group : CHUNKS;
    row.add(c0, c1);
    __syncthreads();
    double *sums = a.sums + static_cast<long>(r) * CHUNKS;
    double v;
    if (gridDim.y > 1) {
        if (wave == 0) {
            if (lane >= c0 && lane < c1)
                __hip_atomic_store(sums + lane, sh.chunk[lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            // The sums are at the agent's coherence point before the workgroup is counted.
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            if (lane == 0)
                arrived = __hip_atomic_fetch_add(a.count_row + r, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (arrived != gridDim.y - 1) return;
        if (t == 0) __hip_atomic_store(a.count_row + r, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        v = __hip_atomic_load(sums + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    } else {
        v = sh.chunk[lane];
    }
    const int token = row.pick(v, u);
    // The sequence that has the row, or where the list is none, each of them.
    for (int b = -1;;) {
        if (t == 0) seq = a.n_seqs;
        __syncthreads();
        for (int i = b + 1 + t; i < a.n_seqs; i += N) {
            const int r0 = a.row0[i], r1 = a.row0[i + 1];
            if (r0 <= r && r < r1 && rows_fit(a, i, r0, r1)) atomicMin(&seq, i);
        }
        __syncthreads();
        b = seq;
        if (b >= a.n_seqs) return;
        const int r0 = a.row0[b], n = a.row0[b + 1] - r0;
        if (t == 0) {
            __hip_atomic_store(a.tokens + r, token, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            arrived = __hip_atomic_fetch_add(a.count + b, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (arrived != static_cast<unsigned>(n) - 1) continue;
        if (t == 0) __hip_atomic_store(a.count + b, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        // Larger trees in the place of their rows' sums, which have been read
        // (all rows are drawn from).
        int *drawn = n <= NODES ? lds : reinterpret_cast<int *>(a.sums + static_cast<long>(r0) * CHUNKS);
        int *first = drawn + n;
        for (int j = t; j < n; j += N) {
            drawn[j] = get(a.tokens + r0 + j);
            first[j] = n;
        }
        __syncthreads();
        // The first child that holds what was drawn at its parent, of each node.
        for (int j = t; j < n; j += N) {
            const int up = a.parent[r0 + j];
            if (up >= 0 && up < j && get(drawn + up) >= 0 && a.draft[r0 + j] == get(drawn + up)) atomicMin(first + up, j);
        }
        __syncthreads();
        // The walk.  Its k-th node takes place k of the list, which is at or
        // before the node's own and not looked at again.  (Sequences that share
        // rows may be walked at once, in the same place: whatever is read back,
        // the walk goes forward, and no node is outside the tree.)
        if (t == 0) {
            int node = 0, kept = 0;
            while (get(drawn + node) >= 0) {
                const int next = get(first + node);
                if (next <= node || next >= n) break;
                first[kept++] = node;
                node = next;
            }
            first[kept] = node;
            if (get(drawn + node) < 0) kept = -1;
            steps = kept;
            a.accepted[b] = kept;
        }
        __syncthreads();
        const int kept = steps;
        for (int j = t; j < n; j += N) {
            int node = j <= kept ? get(first + j) : -1;
            if (node < 0 || node >= n) node = -1;
            a.tokens[r0 + j] = node < 0 ? -1 : get(drawn + node);
            a.path[r0 + j] = node;
        }
        __syncthreads();
    }
}

template <int DT>
hipError_t run(const VerifyTreeArgs &a, hipStream_t st) {
    constexpr int MANY = 1024, FEW = 256;
    if (a.group == 0) {
        k_verify_walk<DT, MANY><<<a.n_seqs, MANY, 0, st>>>(a);
    } else {
        const dim3 grid(a.n_rows > a.n_seqs ? a.n_rows : a.n_seqs, (CHUNKS + a.group - 1) / a.group);
        if (a.few)
            k_verify_rows<DT, FEW><<<grid, FEW, 0, st>>>(a);
        else
            k_verify_rows<DT, MANY><<<grid, MANY, 0, st>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify_tree(const VerifyTreeArgs &args, int dtype, hipStream_t st) {
    VerifyTreeArgs a = args;
    a.segments = (a.vocab + CHUNKS * SEGMENT - 1) / (CHUNKS * SEGMENT);
    // All rows at once, or one after the other as the walk comes by them?  In
    // us, as measured: the first by the bytes and the rows (64 trees of 16 over
    // 32000 fp32 entries: 31; 200: 81; 256 over 32000 in bf16: 63; 250 over 5000
    // in fp16: 25), the second by what the longest of the walks may come by,
    // some six rows (32; 41; 37; 33).  One tree of 32 over 32000: 9 or 13.
    // The drafts' quality is not known here.  Six rows is what drawn trees come
    // by; where more are kept, the walk is chosen all the same and takes longer:
    // 128 chains of 32 over 131072 16-bit entries 73 us with 5 drafts kept, 251
    // with 16, 464 with 31, all rows at once 207 (64 of 32 over 32000 in fp32:
    // 31, 81, 150; 51 to 56).  Where none is kept it is the other way: 64 of 16
    // over 131072 take 56 at once and would walk in 12.
    const double mb = 1e-6 * a.n_rows * static_cast<double>(a.vocab) * (dtype == DT_F32 ? 4 : 2);
    const double rows = 6.0 + mb / 5.5 + 0.0032 * a.n_rows;
    const double levels = a.n_rows < 6 * static_cast<double>(a.n_seqs) ? static_cast<double>(a.n_rows) / a.n_seqs : 6.0;
    const double walk = (8.0 + levels * (2.0 + 7e-5 * a.vocab)) * ((a.n_seqs + 511) / 512);
    a.group = 0;
    if (a.n_rows <= VERIFY_TREE_ROWS && rows <= walk) {
        // Many rows: small workgroups, eight a CU, whose loads and ends overlap
        // (1600 rows of 8000: 18 us instead of 28; 256 of 32000: 16.5 instead
        // of 14.6); of long rows two a row (960 of 100000: 45 instead of 53,
        // 610 of 131072: 41 instead of 58).
        // Few and long ones: up to four large workgroups a row (32 of 131072:
        // 10 us instead of 15; 256: 33 instead of 31).
        a.few = a.n_rows >= 512 || a.vocab <= 4096;
        const int wgs = a.vocab <= 65536 ? 1 : a.few ? 2 : a.n_rows > 128 ? 1 : a.n_rows > 64 ? 2 : 4;
        a.group = CHUNKS / wgs;
    }
    switch (dtype) {
        case DT_F32: return run<DT_F32>(a, st);
        case DT_F16: return run<DT_F16>(a, st);
        default: return run<DT_BF16>(a, st);
    }
}

}  // namespace lora
