// What the training operators launch, checked on the host: their sources are
// compiled for the host alone, the HIP runtime is replaced by the functions
// below, and every entry point is called with addresses that stand for buffers
// of the sizes a caller would give.  For each launch the range that its kernel
// may read or write of every buffer is worked out from its arguments, its tile
// and its grid, and has to lie inside the buffer.  What it reads of the workspace
// must have been written before, as one part, and parts must not overlap.  No
// memory is touched, no GPU needed.
#include "../../draft_verification_row_amd/csrc/embedding.hip"
#include "../../draft_verification_row_amd/csrc/gated.hip"
#include "../../draft_verification_row_amd/csrc/cross_entropy.hip"

#include <cxxabi.h>
#include <stdio.h>
#include <stdlib.h>

#include <iterator>
#include <map>
#include <string>
#include <vector>

// ---------------------------------------------------------------- the buffers
struct Buffer {
    std::string name;
    uintptr_t base;
    size_t bytes;
};
static std::vector<Buffer> buffers;
static std::string call;  // what is being called, for messages
static int failures = 0;
static long launches = 0;
static void fail(const std::string& what) {
    if (++failures <= 40) fprintf(stderr, "%s: %s\n", call.c_str(), what.c_str());
}
static void begin(const std::string& name) {
    buffers.clear();
    call = name;
}
template <typename P>
static P* buffer(const char* name, size_t bytes, int off = 0) {
    const uintptr_t base = ((uintptr_t)buffers.size() + 1) << 42;
    buffers.push_back({name, base + off, bytes});
    return reinterpret_cast<P*>(base + off);
}
// what was written of the workspace in this call: a part's first and last byte
static std::map<std::string, std::pair<uintptr_t, uintptr_t>> parts;
// The buffer of a range, which has to lie inside it.
static const Buffer* range(const char* what, const void* p, long long bytes) {
    if (!p || bytes <= 0) return nullptr;
    const uintptr_t a = (uintptr_t)p, i = a >> 42;
    if (i < 1 || i > buffers.size()) return fail(std::string(what) + " is no buffer"), nullptr;
    const Buffer& b = buffers[i - 1];
    if (a < b.base || a + (uintptr_t)bytes > b.base + b.bytes)
        fail(std::string(what) + " passes the end of " + b.name + " by " + std::to_string((long long)(a + bytes - b.base - b.bytes)) + " bytes");
    return &b;
}
static void writes(const char* part, const void* p, long long bytes) {
    const Buffer* b = range(part, p, bytes);
    if (!b || b->name != "workspace") return;
    const uintptr_t a = (uintptr_t)p;
    auto& r = parts.insert({part, {a, a + bytes}}).first->second;
    if (a < r.first) r.first = a;
    if (a + bytes > r.second) r.second = a + bytes;
}
// slack: read after them and not used
static void reads(const char* what, const void* p, long long bytes, long long slack = 0) {
    const Buffer* b = range(what, p, bytes + slack);
    if (!b || b->name != "workspace") return;
    const uintptr_t a = (uintptr_t)p;
    for (auto& r : parts)
        if (r.second.first <= a && a + bytes <= r.second.second) return;
    fail(std::string(what) + " is read where nothing was written");
}
static long long pad_rows_done, pad_rows_asked;
static size_t most_dz = ~(size_t)0;  // its bytes in this call
static void finish(spec_status s) {
    if (s != SPEC_OK) fail("returned " + std::to_string((int)s));
    for (auto a = parts.begin(); a != parts.end(); ++a)
        for (auto b = std::next(a); b != parts.end(); ++b)
            if (a->second.first < b->second.second && b->second.first < a->second.second) fail(a->first + " overlaps " + b->first);
    if (pad_rows_done < pad_rows_asked) fail("rows left out of the padding");
    pad_rows_done = pad_rows_asked = 0;
    // what the header says of the cross entropy's workspace
    for (auto& p : parts)
        if ((p.first == "dz" && p.second.second - p.second.first > most_dz) || (p.first == "logits" && p.second.second - p.second.first > 1u << 30)) fail(p.first + " take " + std::to_string(p.second.second - p.second.first) + " bytes");
    parts.clear();
}

// --------------------------------------------------------------- the launches
static long long rows_in_all;  // of x and the tokens, as the entry point got them
static long long stats_tiles;  // of the last product with Stats
static std::map<const void*, std::string> names;
template <typename V>
static const V& arg(void** args, int i) { return *static_cast<const V*>(args[i]); }
static long long up(long long x, long long a) { return (x + a - 1) / a * a; }

struct Shape8 {
    int e, bm, bn, wm, wn;  // e: bytes an element
    bool xk, wk, pair, direct;
};
static Shape8 shape_in(const std::string& n) {
    Shape8 s{};
    char type[64], xk[8], wk[8], pair[8], direct[8];
    int stages;
    const size_t at = n.find("Tile<");
    if (at == std::string::npos ||
        sscanf(n.c_str() + at, "Tile<%63[^,], %d, %d, %d, %d, %d, %7[^,], %7[^,], %7[^,], %7[^,]", type, &s.bm, &s.bn, &s.wm, &s.wn, &stages, xk, wk, pair, direct) != 10) {
        fail("no tile in " + n);
        return s;
    }
    s.e = std::string(type) == "float" ? 4 : 2;
    s.xk = xk[0] == 't', s.wk = wk[0] == 't', s.pair = pair[0] == 't', s.direct = direct[0] == 't';
    return s;
}
static int element(const std::string& n) { return n.find("<float") != std::string::npos ? 4 : 2; }
static void outputs(const Outputs& o) {
    writes("loss", o.loss, rows_in_all * 4), writes("lse", o.lse, rows_in_all * 4), writes("status", o.status, rows_in_all * 4), writes("stats", o.stats, rows_in_all * 8);
}
static void weights(const Weights& w) {
    reads("stats", w.stats, rows_in_all * 8), reads("grad loss", w.g_loss, rows_in_all * 4), reads("grad lse", w.g_lse, rows_in_all * 4);
}

static void product(const std::string& n, unsigned grid, void** args) {
    const Product& g = arg<Product>(args, 0);
    const Shape8 s = shape_in(n);
    if (!s.e) return;
    const long long columns = s.pair ? s.bn / 2 : s.bn, tiles_m = (g.M + s.bm - 1) / s.bm, tiles_n = (g.N + columns - 1) / columns;
    const long long splits = g.more > g.splits ? g.more : g.splits, chunk = 16 / s.e, waves_m = s.bm / s.wm;
    if (grid < tiles_m * tiles_n * g.splits * g.products) fail("grid below its tiles: " + n);
    auto operand = [&](const char* what, const void* p, long long ld, bool by_k, long long rows, long long k) {
        if (k > 0) reads(what, p, (by_k ? (k - 1) * ld + rows : (rows - 1) * ld + k) * s.e, by_k && s.direct ? (up(rows, chunk) - rows) * s.e : 0);
    };
    operand("x", g.x[0], g.ldx, s.xk, g.M, g.K), operand("w", g.w[0], g.ldw, s.wk, g.N, g.K);
    if (g.products == 2) operand("the second x", g.x[1], g.ldx, s.xk, g.M, g.K);
    if (s.pair) operand("the second w", g.w[1], g.ldw, s.wk, g.N, g.K);
    if (g.K2) operand("the second x", g.x[1], g.ldx, s.xk, g.M, g.K2), operand("the second w", g.w[1], g.ldw, s.wk, g.N, g.K2);
    reads("count", g.live_m, 4), reads("count", g.live_k, 4);
    const void* e = args[1];
    if (n.find("Store<") != std::string::npos) {
        const long long size = n.find("Store<float") != std::string::npos ? 4 : 2;
        auto& st = *static_cast<const Store<float>*>(e);  // of either type alike
        // the gated block's gradients are done one after the other in one place
        const char* part = call.find("gated") == 0 ? "sums" : s.xk ? "sums of dw" : s.wk ? "sums of dx" : "logits";
        for (int p = 0; p < g.products; ++p) writes(part, st.out[p], ((splits - 1) * st.splits + (g.M - 1) * st.ld + g.N) * size);
    } else if (n.find("GateSums") != std::string::npos) {
        writes("sums", static_cast<const GateSums*>(e)->part, splits * 2 * g.M * g.N * 4);
    } else if (n.find("Gate<") != std::string::npos) {
        auto& o = *static_cast<const Gate<float>*>(e);
        writes("y", o.y, (long long)g.M * g.N * s.e), writes("g", o.g, (long long)g.M * g.N * 4), writes("u", o.u, (long long)g.M * g.N * 4);
    } else if (n.find("Stats<") != std::string::npos) {
        auto& o = *static_cast<const Stats<float>*>(e);
        if (o.v0 % columns) fail("a launch inside a tile");
        stats_tiles = o.v0 / columns + tiles_n;
        reads("tokens", o.tokens, rows_in_all * 4), reads("live", o.live, g.M * 4);
        writes("parts of rows", o.part, ((tiles_n - 1) * o.rows + g.M) * (long long)sizeof(MaxSum)), writes("picked", o.picked, g.M * 4ll);
        reads("bias", o.bias, (long long)g.N * s.e);
    } else if (n.find("Slope<") != std::string::npos) {
        auto& o = *static_cast<const Slope<float>*>(e);
        reads("tokens", o.tokens, rows_in_all * 4), reads("live", o.live, g.M * 4ll), weights(o.weights);
        writes("dz", o.dz, ((g.M - 1) * o.ld + up(g.N, 4)) * s.e), reads("bias", o.bias, (long long)g.N * s.e);
        // a row of sums for every wave row of the grid
        writes("parts of columns", o.part, ((tiles_m * waves_m - 1) * o.V + o.v0 + g.N) * 4);
    } else {
        fail("unknown epilogue: " + n);
    }
}

static void launch(const std::string& n, unsigned grid, unsigned block, void** args) {
    ++launches;
    auto is = [&](const char* kernel) { return n.find(std::string("::") + kernel + "<") != std::string::npos || n.find(std::string("::") + kernel + "(") != std::string::npos; };
    const long long e = element(n);
    if (is("k_product") || is("k_wide")) {
        product(n, grid, args);
    } else if (is("k_lookup")) {
        auto& a = arg<Lookup>(args, 0);
        reads("weight", a.weight, (long long)a.V * a.H * e), reads("tokens", a.tokens, a.n * 4ll), writes("y", a.out, (long long)a.n * a.H * e);
        if ((long long)grid * (block / a.lanes) < a.n) fail("grid below its rows");
    } else if (is("k_rank")) {
        const long long rows = arg<int>(args, 1);
        reads("tokens", arg<const void*>(args, 0), rows * 4), writes("sorted", arg<const void*>(args, 2), rows * 4), writes("position", arg<const void*>(args, 3), rows * 4);
        if (grid * 64ll < rows) fail("grid below its rows");
    } else if (is("k_starts")) {
        reads("sorted", arg<const void*>(args, 0), arg<int>(args, 1) * 4ll), writes("start", arg<const void*>(args, 3), (arg<int>(args, 2) + 1ll) * 4);
        if ((long long)grid * block < arg<int>(args, 2) + 1ll) fail("grid below its tokens");
    } else if (is("k_runs") || is("k_table_grad")) {
        auto& a = arg<TableGrad>(args, 0);
        reads("grad y", a.dy, (long long)a.n * a.H * e), reads("sorted", a.sorted, a.n * 4ll), reads("position", a.position, a.n * 4ll);
        const long long runs = (long long)(a.n / kRun) * a.H * 4;
        if (is("k_runs")) {
            writes("runs", a.part, runs);
            if ((long long)grid * kRun > a.n) fail("grid past its runs");
        } else {
            reads("runs", a.part, runs), reads("start", a.start, (a.V + 1ll) * 4), writes("grad weight", a.out, (long long)a.V * a.H * e);
            if ((long long)grid * kRowsEach * (block / a.lanes) < a.V) fail("grid below its rows");
        }
    } else if (is("k_gated_few")) {
        const Product& g = arg<Product>(args, 0);
        auto& o = arg<Gate<float>>(args, 1);
        reads("x", g.x[0], ((g.M - 1) * g.ldx + g.K) * e), reads("w", g.w[0], ((g.N - 1) * g.ldw + g.K) * e), reads("w of the second", g.w[1], ((g.N - 1) * g.ldw + g.K) * e);
        writes("y", o.y, (long long)g.M * g.N * e), writes("g", o.g, (long long)g.M * g.N * 4), writes("u", o.u, (long long)g.M * g.N * 4);
        if (g.M > 16 || grid * 16ll < g.N) fail("grid below its columns");
    } else if (is("k_gated_join")) {
        const long long M = arg<int>(args, 2), N = arg<int>(args, 3);
        auto& o = arg<Gate<float>>(args, 4);
        reads("sums", arg<const void*>(args, 0), arg<int>(args, 1) * 2 * M * N * 4);
        writes("y", o.y, M * N * e), writes("g", o.g, M * N * 4), writes("u", o.u, M * N * 4);
        if ((long long)grid * block < M * ((N + 3) / 4)) fail("grid below its outputs");
    } else if (is("k_gated_slopes")) {
        auto& a = arg<GateSlope>(args, 0);
        const long long in = (long long)a.M * a.N, out = a.M * a.ld;
        reads("grad y", a.dy, in * e), reads("g", a.g, in * 4), reads("u", a.u, in * 4), writes("dz", a.dg, out * e), writes("dz of the second", a.du, out * e);
        if ((long long)grid * block < a.M * (a.ld / 4)) fail("grid below its outputs");
    } else if (is("k_pad_rows")) {
        auto& a = arg<Pads>(args, 0);
        const long long K = arg<int>(args, 1), ld = arg<int64_t>(args, 2);
        const char* what[3] = {"x", "w", "w of the second"};
        for (int i = 0; i < 3; ++i) {
            const long long rows = a.end[i] - (i ? a.end[i - 1] : 0);
            if (rows) reads(what[i], a.from[i], rows * K * e), writes(what[i], a.to[i], rows * ld * e);
        }
        // launches of some of the rows each
        const long long first = arg<int64_t>(args, 3);
        if (first > pad_rows_done) fail("rows left out of the padding");
        pad_rows_done = first + (long long)grid * block / (ld / (16 / e));
        pad_rows_asked = a.end[2];
    } else if (is("k_join")) {
        const Live& live = arg<Live>(args, 4);
        const long long s = live.count && live.more > arg<int>(args, 1) ? live.more : arg<int>(args, 1), M = arg<int>(args, 5), N = arg<int>(args, 6);
        reads("split sums", arg<const void*>(args, 0), ((s - 1) * arg<int64_t>(args, 2) + M * N) * 4);
        reads("place", arg<const void*>(args, 3), M * 4), reads("count", live.count, 4), writes("joined", arg<const void*>(args, 7), M * N * e);
        if ((long long)grid * block < M * ((N + 3) / 4)) fail("grid below its outputs");
    } else if (is("k_live")) {
        auto& a = arg<Rows>(args, 0);
        reads("tokens", a.tokens, a.M * 4ll), writes("live", a.live, a.M * 4ll), writes("place", a.place, a.M * 4ll), writes("count", a.count, 4), outputs(a.out);
    } else if (is("k_pack")) {
        const long long rows = arg<int64_t>(args, 3), K = arg<int>(args, 4), ld = arg<int64_t>(args, 5);
        const bool live = arg<const void*>(args, 1);
        reads("live", arg<const void*>(args, 1), rows * 4), reads("count", arg<const void*>(args, 2), live ? 4 : 0);
        reads(live ? "x" : "w", arg<const void*>(args, 0), rows * K * e), writes(live ? "x" : "w", arg<const void*>(args, 6), rows * ld * e);
        if ((long long)grid * block < rows * (ld / (16 / e))) fail("grid below its rows");
    } else if (is("k_fold")) {
        auto& a = arg<Fold>(args, 0);
        reads("parts of rows", a.part, (long long)a.parts * a.M * (long long)sizeof(MaxSum)), reads("picked", a.picked, a.M * 4ll);
        reads("tokens", a.tokens, a.M * 4ll), reads("live", a.live, a.M * 4ll), reads("count", a.count, 4), outputs(a.out);
        if (a.parts != stats_tiles) fail("folds other tiles than were written");
        if ((long long)grid * a.across < a.M || kLiveThreads % a.across) fail("grid below its rows");
    } else if (is("k_small_stats") || is("k_small_slope")) {
        auto& a = arg<Small>(args, 0);
        reads("logits", a.part, (long long)a.splits * a.M * a.V * 4), reads("tokens", a.tokens, a.M * 4ll), reads("live", a.live, a.M * 4ll), reads("count", a.count, 4);
        reads("bias", a.bias, a.V * e);
        if (is("k_small_stats")) {
            outputs(arg<Outputs>(args, 1));
        } else {
            weights(arg<Weights>(args, 1));
            writes("dz", arg<const void*>(args, 2), ((a.M - 1) * arg<int64_t>(args, 3) + a.V) * e);
        }
        if (grid < (unsigned)a.M) fail("grid below its rows");
    } else if (is("k_bias_fold")) {
        const Tiling& t = arg<Tiling>(args, 2);
        const long long V = arg<int>(args, 3), rows = (rows_in_all + t.bm - 1) / t.bm * t.waves_m;
        reads("parts of columns", arg<const void*>(args, 0), rows * V * 4), reads("count", arg<const void*>(args, 1), 4), writes("grad bias", arg<const void*>(args, 4), V * e);
        if (grid * 64ll < V) fail("grid below its columns");
    } else {
        fail("unknown kernel: " + n);
    }
}

// ---------------------------------------------------- in the runtime's place
static dim3 grid_, block_;
extern "C" {
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t, hipStream_t) { return grid_ = g, block_ = b, hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3* g, dim3* b, size_t* shared, hipStream_t* st) { return *g = grid_, *b = block_, *shared = 0, *st = nullptr, hipSuccess; }
hipError_t hipLaunchKernel(const void* f, dim3 g, dim3 b, void** args, size_t, hipStream_t) {
    // the hardware counts a launch's threads in 32 bits
    if (g.y != 1 || g.z != 1 || b.y != 1 || b.z != 1 || g.x < 1 || (uint64_t)g.x * b.x >> 32) fail("grid of " + std::to_string(g.x) + ", " + names[f]);
    launch(names[f], g.x, b.x, args);
    return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
void** __hipRegisterFatBinary(const void*) { return nullptr; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipRegisterFunction(void**, const void* f, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
    int bad = 0;
    char* s = abi::__cxa_demangle(name, nullptr, nullptr, &bad);
    names[f] = s ? s : name;
    free(s);
}
}

// ------------------------------------------------------------------ the calls
static std::string title(const char* op, spec_dtype dt, long long a, long long b, long long c, int off) {
    return std::string(op) + " " + (dt == SPEC_BF16 ? "bf16 " : "fp32 ") + std::to_string(a) + " x " + std::to_string(b) + " x " + std::to_string(c) + (off ? " off" : "");
}
static void embedding_calls(spec_dtype dt, int n, int V, int H, int off) {
    const size_t e = elem(dt);
    most_dz = ~(size_t)0;
    begin(title("embedding", dt, n, V, H, off));
    auto* w = buffer<void>("weight", (size_t)V * H * e, off);
    auto* tok = buffer<int32_t>("tokens", n * 4ull);
    finish(spec_embedding(w, dt, tok, 1.f, n, V, H, buffer<void>("y", (size_t)n * H * e, off), nullptr));
    auto* gy = buffer<void>("grad y", (size_t)n * H * e, off);
    auto* gw = buffer<void>("grad weight", (size_t)V * H * e, off);
    const size_t need = spec_embedding_grad_workspace_bytes(dt, n, V, H);
    finish(spec_embedding_grad(tok, gy, dt, 1.f, n, V, H, gw, buffer<void>("workspace", need), need, nullptr));
}
static void gated_calls(spec_dtype dt, int M, int N, int K, int off, bool forward_only = false) {
    most_dz = ~(size_t)0;
    const size_t e = elem(dt), x_ = (size_t)M * K * e, w_ = (size_t)N * K * e, y_ = (size_t)M * N * e, f_ = (size_t)M * N * 4;
    for (int keep = 0; keep < 2; ++keep) {
        begin(title("gated", dt, M, N, K, off));
        rows_in_all = M;
        auto *x = buffer<void>("x", x_, off), *g = buffer<void>("gate", w_, off), *u = buffer<void>("up", w_, off);
        auto *pg = buffer<float>("g", f_), *pu = buffer<float>("u", f_);
        const size_t need = spec_gated_linear_workspace_bytes(dt, M, N, K);
        finish(spec_gated_linear(x, g, u, dt, SPEC_ACT_SILU, M, N, K, buffer<void>("y", y_, off), keep ? pg : nullptr, keep ? pu : nullptr,
                                 buffer<void>("workspace", need), need, nullptr));
    }
    if (forward_only) return;
    for (int which = 1; which < 8; ++which) {
        begin(title("gated gradients", dt, M, N, K, off));
        rows_in_all = M;
        auto *x = buffer<void>("x", x_, off), *g = buffer<void>("gate", w_, off), *u = buffer<void>("up", w_, off);
        auto *pg = buffer<float>("g", f_), *pu = buffer<float>("u", f_);
        auto* gy = buffer<void>("grad y", y_, off);
        auto *gx = buffer<void>("grad x", x_, off), *gg = buffer<void>("grad gate", w_, off), *gu = buffer<void>("grad up", w_, off);
        const size_t need = spec_gated_linear_grad_workspace_bytes(dt, M, N, K);
        finish(spec_gated_linear_grad(x, g, u, pg, pu, gy, dt, SPEC_ACT_SILU, M, N, K, which & 1 ? gx : nullptr, which & 2 ? gg : nullptr,
                                      which & 4 ? gu : nullptr, buffer<void>("workspace", need), need, nullptr));
    }
}
// off: of W alone, or of all operands
static void entropy_calls(spec_dtype dt, int M, int V, int K, int off, bool all_off, bool forward_only = false) {
    const size_t e = elem(dt), x_ = (size_t)M * K * e, w_ = (size_t)V * K * e;
    begin(title("cross entropy", dt, M, V, K, off));
    rows_in_all = M;
    most_dz = M * 1024ull * e > 512 << 20 ? M * 1024ull * e : 512 << 20;
    auto *x = buffer<void>("x", x_, all_off ? off : 0), *w = buffer<void>("weight", w_, off), *b = buffer<void>("bias", V * e, all_off ? off : 0);
    auto* tok = buffer<int32_t>("tokens", M * 4ull);
    auto* stats = buffer<float>("stats", M * 8ull);
    auto *loss = buffer<float>("loss", M * 4ull), *lse = buffer<float>("lse", M * 4ull);
    const size_t need = spec_cross_entropy_workspace_bytes(dt, M, V, K);
    auto* status = buffer<int32_t>("status", M * 4ull);
    finish(spec_cross_entropy(x, w, b, dt, tok, M, V, K, loss, lse, status, stats, buffer<void>("workspace", need), need, nullptr));
    if (forward_only) return;
    const size_t back = spec_cross_entropy_grad_workspace_bytes(dt, M, V, K);
    for (int which = 1; which < 8; ++which) {
        begin(title("cross entropy gradients", dt, M, V, K, off));
        x = buffer<void>("x", x_, all_off ? off : 0), w = buffer<void>("weight", w_, off), b = buffer<void>("bias", V * e, all_off ? off : 0);
        tok = buffer<int32_t>("tokens", M * 4ull), stats = buffer<float>("stats", M * 8ull);
        auto *gl = buffer<float>("grad loss", M * 4ull), *ge = buffer<float>("grad lse", M * 4ull);
        auto *gx = buffer<void>("grad x", x_, all_off ? off : 0), *gw = buffer<void>("grad weight", w_, all_off ? off : 0), *gb = buffer<void>("grad bias", V * e);
        finish(spec_cross_entropy_grad(x, w, b, dt, tok, stats, gl, ge, M, V, K, which & 1 ? gx : nullptr, which & 2 ? gw : nullptr,
                                       which & 4 ? gb : nullptr, buffer<void>("workspace", back), back, nullptr));
    }
}

int main() {
    const int rows[] = {1, 2, 5, 6, 16, 17, 31, 32, 33, 63, 64, 65, 77, 80, 96, 97, 128, 129, 130, 160, 161, 192, 193, 200, 257, 300, 1001, 2050};
    const int columns[] = {1, 7, 64, 72, 129, 700, 4096, 8192, 16000, 32001, 50257};
    const int lengths[] = {1, 3, 64, 72, 200, 515, 768, 777, 1024, 4096};
    for (spec_dtype dt : {SPEC_BF16, SPEC_F32})
        for (int M : rows)
            for (int N : columns)
                for (int K : lengths)
                    for (int off : {0, (int)elem(dt)}) {
                        entropy_calls(dt, M, N, K, off, false);
                        if (off) entropy_calls(dt, M, N, K, off, true);
                        gated_calls(dt, M, N, K, off);
                        embedding_calls(dt, M, N, K, off);
                    }
    // large ones; the vocabulary in pieces, whole and ragged
    for (spec_dtype dt : {SPEC_BF16, SPEC_F32}) {
        for (int V : {128256, 50001, 33000, 262144}) entropy_calls(dt, 8192, V, 64, 0, false), entropy_calls(dt, 8191, V, 1023, 0, false), entropy_calls(dt, 32768, V, 72, (int)elem(dt), true);
        gated_calls(dt, 8192, 14336, 4096, 0), gated_calls(dt, 8191, 14337, 4095, 0), gated_calls(dt, 100000, 24, 16, 0), gated_calls(dt, 70, 90, 50001, 0);
        embedding_calls(dt, 1 << 20, 128256, 4096, 0), embedding_calls(dt, 32768, 1 << 20, 8191, 0), embedding_calls(dt, 1, 1, 1 << 20, 0);
    }
    // long sums of many logits, which are split
    for (spec_dtype dt : {SPEC_BF16, SPEC_F32})
        for (int M : {50, 203, 1061, 5111, 8475, 20654, 36838})
            for (int V : {379, 2615, 4452, 14023, 81876})
                for (int K : {4096, 8192, 16384, 52288, 65536}) entropy_calls(dt, M, V, K, 0, false);
    // the largest that are taken: 2^20 a size, and what the products allow
    const int most = 1 << 20;
    for (spec_dtype dt : {SPEC_BF16, SPEC_F32})
        for (int off : {0, (int)elem(dt)})
            for (int a : {1, 17, 65, 8191, 65535, 262144, most})
                for (int b : {1, 31, 4097, 65536, 262143, most})
                    for (int c : {1, 3, 64, 1023, 8189, 65535, most}) {
                        if (spec_embedding_grad_workspace_bytes(dt, a, b, c)) embedding_calls(dt, a, b, c, off);
                        if (spec_gated_linear_workspace_bytes(dt, a, b, c)) gated_calls(dt, a, b, c, off);
                        if (spec_cross_entropy_workspace_bytes(dt, a, b, c)) entropy_calls(dt, a, b, c, off, true);
                    }
    printf("%ld launches, %d failures\n", launches, failures);
    return failures != 0;
}
