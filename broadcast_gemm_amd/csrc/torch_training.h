// torch_training.h -- the binding of attention's training and of dropout (training.py), included by torch_history.cpp,
// whose checks it uses.
#pragma once

struct TrainingEntry {
    int64_t (*workspace)(int, int, int, int, int, int, int, int);
    int (*forward)(const ikbo_attention_args *, void *);
    int (*backward)(const ikbo_attention_args *, void *);
    int (*dropout)(const ikbo_dropout_args *, void *);
} tr;

void bind_training(const std::vector<uintptr_t> &at) {
    TORCH_CHECK(at.size() == 4, "four entry points");
    tr.workspace = reinterpret_cast<decltype(tr.workspace)>(at[0]);
    tr.forward = reinterpret_cast<decltype(tr.forward)>(at[1]);
    tr.backward = reinterpret_cast<decltype(tr.backward)>(at[2]);
    tr.dropout = reinterpret_cast<decltype(tr.dropout)>(at[3]);
}

void heads4(const char *name, const Tensor &t, const at::Device &d) {
    if (t.scalar_type() != at::kBFloat16 || t.device() != d || t.dim() != 4 || (t.size(3) > 1 && t.stride(3) != 1))
        bad(name, "must be a bfloat16 tensor of four dimensions with contiguous heads, on the device of the others");
}
int64_t stride_of(const Tensor &t, int i) { return t.size(i) > 1 ? t.stride(i) : 0; }

// What both directions take; status of a shape that does not fit, or IKBO_OK.
int attention_args(ikbo_attention_args &a, const Tensor &Q, const Tensor &K, const Tensor &V, const Tensor &map, const Tensor &status, const Maybe &lens,
                   const Maybe &positions, double scale, double dropout, const Maybe &rng, bool backward) {
    const at::Device d = Q.device();
    heads4("Q", Q, d);
    heads4("K", K, d);
    heads4("V", V, d);
    ints("map", map, d);
    status_word(status, d);
    if (lens) ints("lens", *lens, d);
    if (positions) ints("positions", *positions, d);
    if (rng && (rng->scalar_type() != at::kLong || rng->device() != d || !rng->is_contiguous() || rng->numel() != 2))
        bad("rng", "must be a contiguous int64 tensor of two elements (seed, offset) on the device of the others");
    if (dropout > 0 && !rng) bad("rng", "is needed for dropout");
    a.B_u = size32("K", K.size(0));
    a.B_c = size32("Q", Q.size(0));
    a.H_q = size32("Q", Q.size(1));
    a.H_kv = size32("K", K.size(1));
    a.L_q = size32("Q", Q.size(2));
    a.L_kv = size32("K", K.size(2));
    a.head_dim = size32("Q", Q.size(3));
    if (K.sizes() != V.sizes() || K.size(3) != Q.size(3) || map.dim() != 1 || map.size(0) != Q.size(0) || (lens && (lens->dim() != 1 || lens->size(0) != K.size(0))) ||
        (positions && (positions->dim() != 2 || positions->size(0) != Q.size(0) || positions->size(1) != Q.size(2))))
        return IKBO_ERR_INVALID_ARG;
    a.scale = (float)scale;
    if (scale > 0 && a.scale < FLT_MIN) a.scale = FLT_MIN;   // not 0, which is the default; the scores are 0 to float32 either way
    a.dropout = dropout;
    a.workspace_bytes = tr.workspace(a.B_u, a.B_c, a.H_q, a.H_kv, a.L_q, a.L_kv, a.head_dim, backward);
    if (a.workspace_bytes < 0) return (int)a.workspace_bytes;
    a.Q = ptr(Q);
    a.K = ptr(K);
    a.V = ptr(V);
    a.map = ptr<int32_t>(map);
    a.lens = ptr<int32_t>(lens);
    a.positions = ptr<int32_t>(positions);
    a.rng = ptr<int64_t>(rng);
    a.status = ptr<uint32_t>(status);
    a.q_cand = stride_of(Q, 0); a.q_head = stride_of(Q, 1); a.q_query = stride_of(Q, 2);
    a.k_user = stride_of(K, 0); a.k_head = stride_of(K, 1); a.k_token = stride_of(K, 2);
    a.v_user = stride_of(V, 0); a.v_head = stride_of(V, 1); a.v_token = stride_of(V, 2);
    return IKBO_OK;
}

py::object attention_forward(uintptr_t stream, const Tensor &Q, const Tensor &K, const Tensor &V, const Tensor &map, const Tensor &status, const Maybe &lens,
                             const Maybe &positions, double scale, double dropout, const Maybe &rng) {
    ikbo_attention_args a{};
    int st = attention_args(a, Q, K, V, map, status, lens, positions, scale, dropout, rng, false);
    if (st != IKBO_OK) return status_of(st);
    const Tensor O = at::empty(Q.sizes(), Q.options());   // dense, whatever Q's strides are
    const Tensor lse = at::empty({Q.size(0), Q.size(1), Q.size(2)}, Q.options().dtype(at::kFloat));
    const Tensor ws = at::empty({a.workspace_bytes}, Q.options().dtype(at::kByte));
    a.O = ptr(O);
    a.lse = ptr<float>(lse);
    a.workspace = ptr(ws);
    a.o_cand = stride_of(O, 0); a.o_head = stride_of(O, 1); a.o_query = stride_of(O, 2);
    st = tr.forward(&a, stream_of(stream));
    if (st != IKBO_OK) return status_of(st);
    return py::make_tuple(O, lse);
}

py::object attention_backward(uintptr_t stream, const Tensor &dO, const Tensor &Q, const Tensor &K, const Tensor &V, const Tensor &O, const Tensor &lse,
                              const Tensor &map, const Tensor &status, const Maybe &lens, const Maybe &positions, double scale, double dropout, const Maybe &rng) {
    ikbo_attention_args a{};
    const at::Device d = Q.device();
    heads4("dO", dO, d);
    heads4("O", O, d);
    if (lse.scalar_type() != at::kFloat || lse.device() != d || !lse.is_contiguous() || lse.dim() != 3) bad("lse", "must be a contiguous float32 tensor of three dimensions");
    int st = attention_args(a, Q, K, V, map, status, lens, positions, scale, dropout, rng, true);
    if (st != IKBO_OK) return status_of(st);
    if (dO.sizes() != Q.sizes() || O.sizes() != Q.sizes() || lse.sizes() != Q.sizes().slice(0, 3)) return status_of(IKBO_ERR_INVALID_ARG);
    const Tensor dQ = at::empty(Q.sizes(), Q.options()), dK = at::empty(K.sizes(), K.options()), dV = at::empty(V.sizes(), V.options());
    const Tensor ws = at::empty({a.workspace_bytes}, Q.options().dtype(at::kByte));
    a.O = ptr(O);
    a.lse = ptr<float>(lse);
    a.dO = ptr(dO);
    a.dQ = ptr(dQ);
    a.dK = ptr(dK);
    a.dV = ptr(dV);
    a.workspace = ptr(ws);
    a.o_cand = stride_of(O, 0); a.o_head = stride_of(O, 1); a.o_query = stride_of(O, 2);
    a.do_cand = stride_of(dO, 0); a.do_head = stride_of(dO, 1); a.do_query = stride_of(dO, 2);
    a.dq_cand = stride_of(dQ, 0); a.dq_head = stride_of(dQ, 1); a.dq_query = stride_of(dQ, 2);
    a.dk_user = stride_of(dK, 0); a.dk_head = stride_of(dK, 1); a.dk_token = stride_of(dK, 2);
    a.dv_user = stride_of(dV, 0); a.dv_head = stride_of(dV, 1); a.dv_token = stride_of(dV, 2);
    st = tr.backward(&a, stream_of(stream));
    if (st != IKBO_OK) return status_of(st);
    return py::make_tuple(dQ, dK, dV);
}

py::object dropout(uintptr_t stream, const Tensor &x, double p, const Tensor &rng, const Maybe &residual, const Maybe &given) {
    const at::Device d = x.device();
    ikbo_dropout_args a{};
    a.dtype = float_type("x", x);
    if (!x.is_contiguous()) bad("x", "must be contiguous");
    if (residual && (residual->scalar_type() != x.scalar_type() || residual->device() != d || !residual->is_contiguous() || residual->sizes() != x.sizes()))
        bad("residual", "must be a contiguous tensor of x's type, shape and device");
    if (rng.scalar_type() != at::kLong || rng.device() != d || !rng.is_contiguous() || rng.numel() != 2)
        bad("rng", "must be a contiguous int64 tensor of two elements (seed, offset) on the device of x");
    if (given && (given->scalar_type() != x.scalar_type() || given->device() != d || !given->is_contiguous() || given->sizes() != x.sizes()))
        bad("out", "must be a contiguous tensor of x's type, shape and device");
    const Tensor y = given ? *given : at::empty(x.sizes(), x.options());
    a.x = ptr(x);
    a.residual = ptr(residual);
    a.y = ptr(y);
    a.rng = ptr<int64_t>(rng);
    a.n = x.numel();
    a.p = p;
    const int st = tr.dropout(&a, stream_of(stream));
    if (st != IKBO_OK) return status_of(st);
    return py::cast(y);
}
