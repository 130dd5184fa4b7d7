// torch_history.cpp -- the binding of the cached user histories (history.py) and of attention's training (training.py,
// torch_training.h): argument checks, outputs and
// workspaces from torch's allocator, and one call of the C ABI each.  A small call is bound by the host,
// and these steps cost about 10 us in Python; here 3.  Host code only; the library's entry points
// are handed over as addresses (bind), so that there is one libikbo.so in the process.
//
// Every function takes the stream handle first; the tensors' device is current.  Wrong types, devices and
// strides raise ValueError; a status that the library returns comes back as an int.
#include <torch/extension.h>

#include <cfloat>

#include "ikbo.h"

namespace {

using at::Tensor;
using Maybe = std::optional<Tensor>;
namespace py = pybind11;

struct Entry {
    int (*tables)(const ikbo_kv_tables_args *, void *);
    int (*rope)(const ikbo_rope_args *, void *);
    int (*write)(const ikbo_kv4_rows_args *, void *);
    int (*read)(const ikbo_kv4_rows_args *, void *);
    int64_t (*workspace)(int, int, int, int, int, int, int);
    int (*attention)(const ikbo_kv4_attention_args *, void *);
} ik;

void bind(const std::vector<uintptr_t> &at) {
    TORCH_CHECK(at.size() == 6, "six entry points");
    ik.tables = reinterpret_cast<decltype(ik.tables)>(at[0]);
    ik.rope = reinterpret_cast<decltype(ik.rope)>(at[1]);
    ik.write = reinterpret_cast<decltype(ik.write)>(at[2]);
    ik.read = reinterpret_cast<decltype(ik.read)>(at[3]);
    ik.workspace = reinterpret_cast<decltype(ik.workspace)>(at[4]);
    ik.attention = reinterpret_cast<decltype(ik.attention)>(at[5]);
}

[[noreturn]] void bad(const char *name, const char *what) { throw py::value_error(std::string(name) + " " + what); }

template <class T = void>
T *ptr(const Tensor &t) { return static_cast<T *>(t.data_ptr()); }
template <class T = void>
T *ptr(const Maybe &t) { return t ? static_cast<T *>(t->data_ptr()) : nullptr; }

int size32(const char *name, int64_t n) {
    if (n > INT32_MAX) bad(name, "is too large");
    return (int)n;
}

void ints(const char *name, const Tensor &t, const at::Device &d) {
    if (t.scalar_type() != at::kInt || t.device() != d || !t.is_contiguous())
        bad(name, "must be a contiguous int32 tensor on the device of the others");
}
void status_word(const Tensor &t, const at::Device &d) {
    if (t.scalar_type() != at::kInt || t.device() != d || t.numel() != 1) bad("status", "must be an int32 tensor of one element");
}
void block_table(const Tensor &t, const at::Device &d) {
    if (t.scalar_type() != at::kInt || t.device() != d || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
        bad("the block table", "must be an int32 tensor [users, pages] with contiguous rows");
}
int float_type(const char *name, const Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return IKBO_DTYPE_BF16;
    if (t.scalar_type() == at::kFloat) return IKBO_DTYPE_F32;
    bad(name, "must be bfloat16 or float32");
}
// Rows [tokens, heads, head_dim] with contiguous heads.
void heads(const char *name, const Tensor &t, const at::Device &d, at::ScalarType type) {
    if (t.scalar_type() != type || t.device() != d || t.dim() != 3 || (t.size(2) > 1 && t.stride(2) != 1))
        bad(name, "must be a tensor [tokens, heads, head_dim] with contiguous heads, of the others' type and device");
}
void check_tiles(const Tensor &t, const at::Device &d) {
    if (t.scalar_type() != at::kByte || t.device() != d || t.dim() != 3 || !t.is_contiguous())
        bad("tiles", "must be a contiguous uint8 tensor [pages, heads, 68 * head_dim]");
}
void *stream_of(uintptr_t s) { return reinterpret_cast<void *>(s); }
py::object status_of(int st) { return py::int_(st); }

// slots, positions, rows, starts, lens_out, state_out; `out` holds them, or lens_out and state_out alone.
py::object kv_tables(uintptr_t stream, const Tensor &counts, const Tensor &lens, const Tensor &table, const Tensor &ring, const Tensor &state,
                     int64_t capacity, const Tensor &status, int64_t page_size, bool in_place, const std::optional<std::vector<Tensor>> &out) {
    const at::Device d = lens.device();
    ints("counts", counts, d);
    ints("lens", lens, d);
    ints("ring", ring, d);
    ints("state", state, d);
    block_table(table, d);
    status_word(status, d);
    const int64_t B = lens.numel();
    if (counts.numel() != B || table.size(0) != B || state.numel() != 4 || capacity < 0) return status_of(IKBO_ERR_INVALID_ARG);
    std::vector<Tensor> t;
    if (out) {
        t = *out;
        if (t.size() != 6) bad("out", "must be the six tensors of a step");
        for (const Tensor &x : t) ints("out", x, d);
        if (t[0].numel() != capacity || t[1].numel() != capacity || t[2].numel() != capacity || t[3].numel() != B + 1 || t[4].numel() != B ||
            t[5].numel() != 4)
            return status_of(IKBO_ERR_INVALID_ARG);
    } else {
        // One allocation for all of them.
        const Tensor all = at::empty({3 * capacity + B + 1 + (in_place ? 0 : B + 4)}, lens.options());
        const int64_t sizes[] = {capacity, capacity, capacity, B + 1, B, 4};
        int64_t at = 0;
        for (int i = 0; i < (in_place ? 4 : 6); ++i) {
            t.push_back(all.narrow(0, at, sizes[i]));
            at += sizes[i];
        }
        if (in_place) {
            t.push_back(lens);
            t.push_back(state);
        }
    }
    ikbo_kv_tables_args a{};
    a.counts = ptr<int32_t>(counts);
    a.lens = ptr<int32_t>(lens);
    a.lens_out = ptr<int32_t>(t[4]);
    a.block_table = ptr<int32_t>(table);
    a.ring = ptr<int32_t>(ring);
    a.state = ptr<int32_t>(state);
    a.state_out = ptr<int32_t>(t[5]);
    a.slots = ptr<int32_t>(t[0]);
    a.positions = ptr<int32_t>(t[1]);
    a.rows = ptr<int32_t>(t[2]);
    a.starts = ptr<int32_t>(t[3]);
    a.status = ptr<uint32_t>(status);
    a.table_stride = table.stride(0);
    a.B_u = size32("lens", B);
    a.max_pages = size32("the block table", table.size(1));
    a.num_pages = size32("ring", ring.numel());
    a.page_size = size32("page_size", page_size);
    a.capacity = size32("capacity", capacity);
    const int st = ik.tables(&a, stream_of(stream));
    if (st != IKBO_OK) return status_of(st);
    return py::make_tuple(t[0], t[1], t[2], t[3], t[4], t[5]);
}

py::object rope(uintptr_t stream, const Maybe &q, const Maybe &k, const Tensor &positions, const Tensor &freq, int layout, double factor,
                bool inverse, const Maybe &q_given, const Maybe &k_given) {
    const Tensor &x = q ? *q : *k;
    const at::Device d = x.device();
    ikbo_rope_args a{};
    a.dtype = float_type("q and k", x);
    if (q) heads("q", *q, d, x.scalar_type());
    if (k) heads("k", *k, d, x.scalar_type());
    ints("positions", positions, d);
    if (freq.scalar_type() != at::kDouble || freq.device() != d || !freq.is_contiguous() || freq.dim() != 1)
        bad("freq", "must be a contiguous float64 tensor [rot_dim / 2]");
    const int64_t T = x.size(0);
    if (positions.dim() != 1 || positions.size(0) != T || (k && (k->size(0) != T || k->size(2) != x.size(2)))) return status_of(IKBO_ERR_INVALID_ARG);
    Maybe qo = q_given, ko = k_given;
    if (q && !qo) qo = at::empty(q->sizes(), x.options());
    if (k && !ko) ko = at::empty(k->sizes(), x.options());
    for (const auto &[in, out] : {std::make_pair(&q, &qo), std::make_pair(&k, &ko)}) {
        if (!*in) continue;
        heads("out", **out, d, x.scalar_type());
        if ((*out)->sizes() != (*in)->sizes()) return status_of(IKBO_ERR_INVALID_ARG);
    }
    if (q) {
        a.q = ptr(*q); a.q_token = q->stride(0); a.q_head = q->stride(1);
        a.q_out = ptr(*qo); a.q_out_token = qo->stride(0); a.q_out_head = qo->stride(1);
        a.H_q = size32("q", q->size(1));
    }
    if (k) {
        a.k = ptr(*k); a.k_token = k->stride(0); a.k_head = k->stride(1);
        a.k_out = ptr(*ko); a.k_out_token = ko->stride(0); a.k_out_head = ko->stride(1);
        a.H_k = size32("k", k->size(1));
    }
    a.positions = ptr<int32_t>(positions);
    a.freq = ptr<double>(freq);
    a.T = size32("q", T);
    a.head_dim = size32("q", x.size(2));
    a.rot_dim = size32("freq", 2 * freq.size(0));
    a.layout = layout;
    a.inverse = inverse;
    a.factor = (float)factor;
    const int st = ik.rope(&a, stream_of(stream));
    if (st != IKBO_OK) return status_of(st);
    return py::make_tuple(qo, ko);
}

ikbo_kv4_rows_args rows_args(const Tensor &k, const Tensor &v, const Tensor &slots, const Tensor &tiles, const Tensor &status) {
    ikbo_kv4_rows_args a{};
    a.k = ptr(k);
    a.v = ptr(v);
    a.slots = ptr<int32_t>(slots);
    a.tiles = ptr(tiles);
    a.status = ptr<uint32_t>(status);
    a.k_token = k.stride(0);
    a.k_head = k.stride(1);
    a.v_token = v.stride(0);
    a.v_head = v.stride(1);
    a.T = size32("slots", slots.numel());
    a.H_kv = size32("tiles", tiles.size(1));
    a.head_dim = size32("tiles", tiles.size(2) / 68);
    a.num_pages = size32("tiles", tiles.size(0));
    return a;
}
bool rows_fit(const Tensor &x, const Tensor &slots, const Tensor &tiles) {
    return x.size(0) == slots.numel() && x.size(1) == tiles.size(1) && tiles.size(2) % 68 == 0 && x.size(2) == tiles.size(2) / 68;
}

int kv4_write(uintptr_t stream, const Tensor &k, const Tensor &v, const Tensor &slots, const Tensor &tiles, const Tensor &status) {
    const at::Device d = k.device();
    const int type = float_type("k and v", k);
    heads("k", k, d, k.scalar_type());
    heads("v", v, d, k.scalar_type());
    ints("slots", slots, d);
    check_tiles(tiles, d);
    status_word(status, d);
    if (!rows_fit(k, slots, tiles) || !rows_fit(v, slots, tiles)) return IKBO_ERR_INVALID_ARG;
    ikbo_kv4_rows_args a = rows_args(k, v, slots, tiles, status);
    a.dtype = type;
    return ik.write(&a, stream_of(stream));
}

py::object kv4_read(uintptr_t stream, const Tensor &slots, const Tensor &tiles, const Tensor &status, at::ScalarType type, const Maybe &k_given,
                    const Maybe &v_given) {
    const at::Device d = tiles.device();
    ints("slots", slots, d);
    check_tiles(tiles, d);
    status_word(status, d);
    if (tiles.size(2) % 68 != 0) return status_of(IKBO_ERR_INVALID_ARG);
    const bool given = k_given.has_value();
    if (!given && type != at::kBFloat16 && type != at::kFloat) bad("dtype", "must be bfloat16 or float32");
    const auto fresh = [&] { return at::empty({slots.numel(), tiles.size(1), tiles.size(2) / 68}, tiles.options().dtype(type)); };
    const Tensor k = given ? *k_given : fresh(), v = given ? *v_given : fresh();
    const int dtype = float_type("out", k);
    heads("out", k, d, k.scalar_type());
    heads("out", v, d, k.scalar_type());
    if (!rows_fit(k, slots, tiles) || !rows_fit(v, slots, tiles)) return status_of(IKBO_ERR_INVALID_ARG);
    ikbo_kv4_rows_args a = rows_args(k, v, slots, tiles, status);
    a.dtype = dtype;
    const int st = ik.read(&a, stream_of(stream));
    if (st != IKBO_OK) return status_of(st);
    return py::make_tuple(k, v);
}

py::object kv4_attention(uintptr_t stream, const Tensor &Q, const Tensor &tiles, const Tensor &table, const Tensor &lens, const Maybe &map,
                         const Tensor &status, const Maybe &positions, double scale, const Maybe &given) {
    const at::Device d = Q.device();
    const int64_t nd = Q.dim();
    if (Q.scalar_type() != at::kBFloat16 || (nd != 3 && nd != 4) || (Q.size(-1) > 1 && Q.stride(-1) != 1))
        bad("Q", "must be a bfloat16 tensor [B_c, H_q, L_q, head_dim] or [B_c, H_q, head_dim] with contiguous heads");
    check_tiles(tiles, d);
    block_table(table, d);
    ints("lens", lens, d);
    status_word(status, d);
    if (map) ints("map", *map, d);
    if (positions) ints("positions", *positions, d);
    const int64_t B_c = Q.size(0), H_q = Q.size(1), L_q = nd == 4 ? Q.size(2) : 1, B_u = lens.numel();
    if (68 * Q.size(-1) != tiles.size(2) || table.size(0) != B_u || (map && (map->dim() != 1 || map->size(0) != B_c)) ||
        (positions && positions->numel() != B_c * L_q))
        return status_of(IKBO_ERR_INVALID_ARG);
    if (given && (given->scalar_type() != at::kBFloat16 || given->device() != d || given->sizes() != Q.sizes() ||
                  (Q.size(-1) > 1 && given->stride(-1) != 1)))
        bad("out", "must be a bfloat16 tensor shaped like Q with contiguous heads");
    ikbo_kv4_attention_args a{};
    a.B_u = size32("lens", B_u);
    a.B_c = size32("Q", B_c);
    a.H_q = size32("Q", H_q);
    a.H_kv = size32("tiles", tiles.size(1));
    a.L_q = size32("Q", L_q);
    a.head_dim = size32("Q", Q.size(-1));
    a.max_pages = size32("the block table", table.size(1));
    a.num_pages = size32("tiles", tiles.size(0));
    a.scale = (float)scale;
    if (scale > 0 && a.scale < FLT_MIN) a.scale = FLT_MIN;   // not 0, which is the default; the scores are 0 to float32 either way
    a.workspace_bytes = ik.workspace(a.B_u, a.B_c, a.H_q, a.H_kv, a.L_q, a.head_dim, a.max_pages);
    if (a.workspace_bytes < 0) return status_of((int)a.workspace_bytes);
    const Tensor O = given ? *given : at::empty(Q.sizes(), Q.options());
    const Tensor ws = at::empty({a.workspace_bytes}, tiles.options());
    a.Q = ptr(Q);
    a.O = ptr(O);
    a.tiles = ptr(tiles);
    a.block_table = ptr<int32_t>(table);
    a.lens = ptr<int32_t>(lens);
    a.map = ptr<int32_t>(map);
    a.positions = ptr<int32_t>(positions);
    a.status = ptr<uint32_t>(status);
    a.workspace = ptr(ws);
    a.q_cand = Q.stride(0);
    a.q_head = Q.stride(1);
    a.q_query = nd == 4 ? Q.stride(2) : 0;
    a.o_cand = O.stride(0);
    a.o_head = O.stride(1);
    a.o_query = nd == 4 ? O.stride(2) : 0;
    a.table_stride = table.stride(0);
    const int st = ik.attention(&a, stream_of(stream));
    if (st != IKBO_OK) return status_of(st);
    return py::cast(O);
}

#include "torch_training.h"

}  // namespace

PYBIND11_MODULE(_ikbo_torch, m) {
    m.def("bind", &bind);
    m.def("kv_tables", &kv_tables);
    m.def("rope", &rope);
    m.def("kv4_write", &kv4_write);
    m.def("kv4_read", &kv4_read);
    m.def("kv4_attention", &kv4_attention);
    m.def("bind_training", &bind_training);
    m.def("attention_forward", &attention_forward);
    m.def("attention_backward", &attention_backward);
    m.def("dropout", &dropout);
}
