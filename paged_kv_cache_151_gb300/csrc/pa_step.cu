// pa_step.cu -- block tables and maps of a step built on the device from the
// requests' lengths, and blocks past a length given back.
//
// "vLLM: Architecture, PagedAttention & Internals", *The free list and the block
// table* (a request holds ceil(n / block_size) blocks; the next token takes a new
// one only when it starts one) and *The forward step in detail* (slot = block *
// block_size + offset), for lengths that only the device knows: behind
// pa_verify_drafts the number of tokens a sequence has grown by is a device array.
//
// Building: sequence s needs need_s = max(ceil((ctx + new) / 16) - held, 0) blocks
// and has new_s rows; two prefix sums over the sequences give its first row and its
// place in the free list, from whose end blocks are taken in the order of the
// sequences.  Trimming is the reverse: the blocks past ceil(keep / 16) go back so
// that the first sequence's first one is taken next.
//
// Bound by latency (a decode batch moves a hundred KB).  One cluster of up to eight
// blocks does everything in one launch, since the state is updated in place: every
// block runs the prefix sums over all sequences itself (they are read once from
// HBM and seven times from L2), then handles a run of the sequences; counts are written
// behind a cluster barrier that every block's reads precede.  A request named twice
// would be given blocks twice, or give them back twice, so every block marks the
// requests in a bit map in shared memory on the way, and nothing is served if a mark
// was there already.  Building a step of 256 sequences with five rows each takes 6 us
// and its trim 6, of 3001 requests with 33649 rows 29 us together: a launch, and one
// after the other the loads of ids, lengths, counts and tables with a cluster's
// barrier, some eight trips to memory.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int ST_THREADS = 1024;
constexpr int ST_WARPS = ST_THREADS / 32;
constexpr int ST_CLUSTER = 8;
// entries of a table that one warp copies; longer tables are shared by the block
constexpr int ST_WARP_ENTRIES = 512;
// sequences that a warp takes side by side
constexpr int SIDE = 4;

__device__ __forceinline__ int blocks_for(int64_t tokens) { return (int)((tokens + 15) >> 4); }

// Exclusive sums of two values over the block's threads, and their totals.
__device__ __forceinline__ void scan2(int64_t &a, int64_t &b, int64_t &ta, int64_t &tb, int64_t (*sh)[ST_WARPS]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    if (lane == 31) {
        sh[0][warp] = x;
        sh[1][warp] = y;
    }
    __syncthreads();
    if (warp == 0) {
        int64_t u = sh[0][lane], v = sh[1][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t uu = __shfl_up_sync(0xffffffffu, u, o), vv = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) {
                u += uu;
                v += vv;
            }
        }
        sh[0][lane] = u;
        sh[1][lane] = v;
    }
    __syncthreads();
    a = x - a + (warp ? sh[0][warp - 1] : 0);
    b = y - b + (warp ? sh[1][warp - 1] : 0);
    ta = sh[0][ST_WARPS - 1];
    tb = sh[1][ST_WARPS - 1];
}

// Words of the map of the requests that a call names.
__host__ __device__ __forceinline__ int map_words(const StepParams &p) {
    return p.request_ids ? (p.num_requests + 31) / 32 : 0;
}

// Whether request `id` is marked already; marks it.
__device__ __forceinline__ bool mark(uint32_t *map, int id) {
    const uint32_t bit = 1u << (id & 31);
    return (atomicOr(&map[id >> 5], bit) & bit) != 0;
}

// What the step wants for sequence s.
struct Want {
    int id, ctx, rows, held;
    bool id_ok;
    int64_t need;                          // blocks to take, -1: a bad id or length
};

__device__ __forceinline__ Want want_of(const StepParams &p, int s) {
    Want w;
    w.id = p.request_ids ? p.request_ids[s] : s;
    w.ctx = p.context_lens[s];
    w.rows = p.new_lens ? p.new_lens[s] : 1;
    w.id_ok = w.id >= 0 && w.id < p.num_requests;
    w.held = w.id_ok ? p.request_blocks[w.id] : 0;
    const int64_t end = (int64_t)w.ctx + w.rows;
    const int width = min(p.max_blocks, p.request_width);
    const bool ok = w.id_ok && w.ctx >= 0 && w.rows >= 0 && end <= (int64_t)width * 16 &&
                    w.held >= 0 && w.held <= p.request_width;
    w.rows = max(w.rows, 0);
    w.need = ok ? max(blocks_for(end) - w.held, 0) : -1;
    return w;
}

// A sequence of this block's run: first row, tokens before it, blocks held (-1: it
// is refused), first place from the free list's end.
struct __align__(16) Seq {
    int row, ctx, held, place;
};

__global__ void __launch_bounds__(ST_THREADS, 1) build_step_kernel(const __grid_constant__ StepParams p) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Seq *seqs = reinterpret_cast<Seq *>(smem_raw);         // [run + 1]
    __shared__ int64_t sh[2][ST_WARPS];
    __shared__ int sh_taken, sh_long, sh_twice;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
    const int B = p.num_seqs;
    const int lo = (int)((int64_t)B * rank / C), hi = (int)((int64_t)B * (rank + 1) / C);
    uint32_t *named = reinterpret_cast<uint32_t *>(seqs + B / C + 2);
    for (int i = tid; i < map_words(p); i += ST_THREADS) named[i] = 0;
    if (tid == 0) sh_taken = sh_long = sh_twice = 0;
    __syncthreads();

    int count = p.free_count ? *p.free_count : 0;
    if (count < 0 || count > p.free_capacity) {
        if (rank == 0 && tid == 0) set_error(p.err, ERR_BLOCK_ID);
        count = count < 0 ? 0 : (int)p.free_capacity;
    }

    // ---- the sums over all sequences, `per` neighbours a thread
    const int per = (B + ST_THREADS - 1) / ST_THREADS;
    const int s0 = min(B, tid * per), s1 = min(B, s0 + per);
    int64_t rows = 0, need = 0, all_rows, all_need;
    for (int s = s0; s < s1; ++s) {
        const Want w = want_of(p, s);
        if (p.request_ids && w.id_ok && mark(named, w.id)) sh_twice = 1;
        rows += w.rows;
        need += w.need > 0 ? w.need : 0;
    }
    scan2(rows, need, all_rows, all_need, sh);
    const bool twice = sh_twice;           // nothing is served
    unsigned bad = twice ? ERR_SEQ_LEN : 0;
    int taken = 0;                         // blocks that the last granted sequence reaches to
    for (int s = s0; s < s1; ++s) {
        const Want w = want_of(p, s);
        const int64_t end = need + (w.need > 0 ? w.need : 0), row_end = rows + w.rows;
        bool ok = w.need >= 0 && row_end <= p.num_rows;
        if (!ok && !(p.request_ids && w.id == -1 && row_end <= p.num_rows)) bad |= ERR_SEQ_LEN;
        ok = ok && !twice;
        if (ok && w.need > 0) {
            if (end <= count) {
                taken = (int)end;
            } else {
                ok = false;
                bad |= ERR_BLOCKS;
            }
        }
        const int row = (int)min(rows, p.num_rows);
        if (s >= lo && s < hi) {
            seqs[s - lo] = Seq{row, w.ctx, ok ? w.held : -1, (int)min(need, (int64_t)INT32_MAX)};
            p.query_start[s] = row;
            p.seq_lens[s] = ok ? w.ctx + w.rows : 0;
            if (ok && blocks_for((int64_t)w.ctx + w.rows) > ST_WARP_ENTRIES) sh_long = 1;
        }
        if (s == hi) seqs[s - lo].row = row;
        need = end;
        rows = row_end;
    }
    if (tid == 0 && hi == B) seqs[hi - lo].row = (int)min(all_rows, p.num_rows);
    if (tid == 0 && rank == 0) p.query_start[B] = (int)min(all_rows, p.num_rows);
    if (bad && rank == 0) set_error(p.err, bad);
    if (taken) atomicMax(&sh_taken, taken);
    if (C > 1) cluster_arrive();           // this block has read the counts
    __syncthreads();

    // entry e of a granted sequence's table
    auto entry = [&](const Seq &q, const int32_t *row, int e) -> int32_t {
        return e < q.held ? row[e] : p.free_blocks[count - 1 - (q.place + e - q.held)];
    };
    auto rows_of = [&](int i) -> int { return seqs[i + 1].row - seqs[i].row; };

    // ---- tables: a warp per sequence; the part past ST_WARP_ENTRIES by the block
    auto table = [&](int i, int e0, int e1, int start, int step) {
        const Seq q = seqs[i];
        const int s = lo + i;
        const int32_t id = p.request_ids ? p.request_ids[s] : s;
        int32_t *req = p.request_tables + (int64_t)id * p.request_width;
        int32_t *out = p.block_tables + (int64_t)s * p.max_blocks;
#pragma unroll 4
        for (int e = e0 + start; e < e1; e += step) {
            const int32_t b = entry(q, req, e);
            out[e] = b;
            if (e >= q.held) req[e] = b;
        }
    };
    // (four sequences' first entries at a time: one after the other each waited for its
    // id and for its table, 33.7 us for 3001 requests where it is 29.3)
    for (int i0 = warp; i0 < hi - lo; i0 += ST_WARPS * SIDE) {
        int n[SIDE], b[SIDE][2];
        int64_t id[SIDE];
#pragma unroll
        for (int j = 0; j < SIDE; ++j) {
            const int i = i0 + j * ST_WARPS;
            const bool some = i < hi - lo && seqs[i].held >= 0;
            n[j] = some ? min(blocks_for((int64_t)seqs[i].ctx + rows_of(i)), ST_WARP_ENTRIES) : 0;
            id[j] = some && p.request_ids ? p.request_ids[lo + i] : lo + i;
        }
#pragma unroll
        for (int j = 0; j < SIDE; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (lane + 32 * h < n[j])
                    b[j][h] = entry(seqs[i0 + j * ST_WARPS], p.request_tables + id[j] * p.request_width, lane + 32 * h);
#pragma unroll
        for (int j = 0; j < SIDE; ++j) {
            const int i = i0 + j * ST_WARPS;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int e = lane + 32 * h;
                if (e >= n[j]) continue;
                p.block_tables[(int64_t)(lo + i) * p.max_blocks + e] = b[j][h];
                if (e >= seqs[i].held) p.request_tables[id[j] * p.request_width + e] = b[j][h];
            }
            if (n[j] > 64) table(i, 64, n[j], lane, 32);
        }
    }
    if (sh_long) {
        for (int i = 0; i < hi - lo; ++i) {
            if (seqs[i].held < 0) continue;
            const int n = blocks_for((int64_t)seqs[i].ctx + rows_of(i));
            if (n > ST_WARP_ENTRIES) table(i, ST_WARP_ENTRIES, n, tid, ST_THREADS);
        }
    }

    // ---- positions and slots of this run's rows
    const int r0 = seqs[0].row, r1 = seqs[hi - lo].row;
    auto place = [&](int r, int64_t &pos, int64_t &slot) {
        int a = 0, b = hi - lo - 1;        // the last sequence that starts at or before r
        while (a < b) {
            const int mid = (a + b + 1) >> 1;
            if (seqs[mid].row <= r) a = mid; else b = mid - 1;
        }
        const Seq q = seqs[a];
        pos = (int64_t)q.ctx + (r - q.row);
        slot = -1;
        if (q.held >= 0) {
            const int s = lo + a;
            const int32_t id = p.request_ids ? p.request_ids[s] : s;
            const int32_t blk = entry(q, p.request_tables + (int64_t)id * p.request_width, (int)(pos >> 4));
            if (blk >= 0 && blk < p.num_blocks) slot = (int64_t)blk * 16 + (pos & 15);
            else set_error(p.err, ERR_BLOCK_ID);
        }
    };
    for (int r = r0 + tid; r < r1 && hi > lo; r += ST_THREADS) {
        int64_t pos, slot;
        place(r, pos, slot);
        p.positions[r] = pos;
        p.slot_mapping[r] = slot;
    }
    // padding behind the last row
    for (int64_t r = min(all_rows, p.num_rows) + rank * ST_THREADS + tid; r < p.num_rows; r += (int64_t)C * ST_THREADS) {
        p.positions[r] = 0;
        p.slot_mapping[r] = -1;
    }

    // ---- the counts, once every block of the cluster has read them
    if (C > 1) cluster_wait();
    for (int i = tid; i < hi - lo; i += ST_THREADS) {
        const Seq q = seqs[i];
        const int n = blocks_for((int64_t)q.ctx + rows_of(i));
        if (q.held >= 0 && n > q.held) p.request_blocks[p.request_ids ? p.request_ids[lo + i] : lo + i] = n;
    }
    if (rank == 0 && tid == 0 && sh_taken > 0) *p.free_count = count - sh_taken;
}

__global__ void __launch_bounds__(ST_THREADS, 1) trim_blocks_kernel(const __grid_constant__ StepParams p) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    int4 *seqs = reinterpret_cast<int4 *>(smem_raw);       // id, kept, given back, place
    __shared__ int64_t sh[2][ST_WARPS];
    __shared__ int sh_twice;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
    const int B = p.num_seqs;
    const int lo = (int)((int64_t)B * rank / C), hi = (int)((int64_t)B * (rank + 1) / C);
    uint32_t *named = reinterpret_cast<uint32_t *>(seqs + B / C + 2);
    for (int i = tid; i < map_words(p); i += ST_THREADS) named[i] = 0;
    if (tid == 0) sh_twice = 0;
    __syncthreads();
    const int count0 = *p.free_count;
    const bool count_ok = count0 >= 0 && count0 <= p.free_capacity;
    const int64_t count = count_ok ? count0 : p.free_capacity;     // nothing fits then
    if (!count_ok && rank == 0 && tid == 0) set_error(p.err, ERR_BLOCK_ID);

    auto back_of = [&](int s, int &id, int &keep) -> int {
        id = p.request_ids ? p.request_ids[s] : s;
        const int len = p.context_lens[s];
        const bool id_ok = id >= 0 && id < p.num_requests;
        const int held = id_ok ? p.request_blocks[id] : 0;
        if (!id_ok || len < 0 || held < 0 || held > p.request_width) {
            keep = p.request_ids && id == -1 ? 0 : -1;
            return 0;
        }
        keep = min(held, blocks_for(len));
        return held - keep;
    };
    const int per = (B + ST_THREADS - 1) / ST_THREADS;
    const int s0 = min(B, tid * per), s1 = min(B, s0 + per);
    int64_t back = 0, none = 0, all_back, all_none;
    for (int s = s0; s < s1; ++s) {
        int id, keep;
        back += back_of(s, id, keep);
        if (p.request_ids && id >= 0 && id < p.num_requests && mark(named, id)) sh_twice = 1;
    }
    scan2(back, none, all_back, all_none, sh);
    bool bad = sh_twice;
    bool fits = count_ok && count + all_back <= p.free_capacity;
    if (!fits && !bad && rank == 0 && tid == 0) set_error(p.err, ERR_BLOCK_ID);
    fits = fits && !bad;                   // a request named twice: nothing changes
    for (int s = s0; s < s1; ++s) {
        int id, keep;
        const int n = back_of(s, id, keep);
        bad = bad || keep < 0;
        if (s >= lo && s < hi) seqs[s - lo] = make_int4(id, keep, n, (int)min(back, (int64_t)INT32_MAX));
        back += n;
    }
    if (bad && rank == 0) set_error(p.err, ERR_SEQ_LEN);
    if (C > 1) cluster_arrive();           // this block has read the counts
    __syncthreads();
    if (fits) {
        for (int i0 = warp; i0 < hi - lo; i0 += ST_WARPS * SIDE) {
            int4 q[SIDE];                  // (side by side, as in the building)
            int32_t b[SIDE];
#pragma unroll
            for (int j = 0; j < SIDE; ++j) {
                const int i = i0 + j * ST_WARPS;
                q[j] = i < hi - lo ? seqs[i] : make_int4(0, 0, 0, 0);
                if (lane < q[j].z) b[j] = p.request_tables[(int64_t)q[j].x * p.request_width + q[j].y + lane];
            }
#pragma unroll
            for (int j = 0; j < SIDE; ++j) {
                const int32_t *req = p.request_tables + (int64_t)q[j].x * p.request_width + q[j].y;
                int32_t *to = p.free_blocks + (count + all_back - 1 - q[j].w);
                if (lane < q[j].z) to[-lane] = b[j];
                for (int e = lane + 32; e < q[j].z; e += 32) to[-e] = req[e];
            }
        }
    }
    if (C > 1) cluster_wait();
    if (!fits) return;
    for (int i = tid; i < hi - lo; i += ST_THREADS)
        if (seqs[i].z > 0) p.request_blocks[seqs[i].x] = seqs[i].y;
    if (rank == 0 && tid == 0) *p.free_count = (int)(count + all_back);
}

// Shared memory of a run's records.
size_t records(const StepParams &p, int C) { return ((size_t)p.num_seqs / C + 2) * 16; }

// Blocks of the cluster: one for every few sequences or thousand rows.
int cluster_of(const StepParams &p) {
    const int64_t work = p.num_rows + 32 * (int64_t)p.num_seqs;
    int C = 1;
    while (C < ST_CLUSTER && work > (int64_t)C * 1024) C *= 2;
    // a run's records have to fit into shared memory
    while (C < ST_CLUSTER && records(p, C) > 40 * 1024) C *= 2;
    return C;
}

template <typename Kernel>
cudaError_t launch(Kernel kern, const StepParams &p, cudaStream_t st) {
    const int C = cluster_of(p);
    const size_t smem = records(p, C) + (size_t)map_words(p) * 4;      // <= 131 + 65 KB
    if (smem > 46 * 1024) {                 // beside the static part
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C, 1, 1);
    cfg.blockDim = dim3(ST_THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t build_step(const StepParams &p, cudaStream_t st) { return launch(build_step_kernel, p, st); }
cudaError_t trim_blocks(const StepParams &p, cudaStream_t st) { return launch(trim_blocks_kernel, p, st); }

}  // namespace pa
