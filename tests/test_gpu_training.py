"""Attention's training and dropout on the GPU against their plain 64-bit forms (training_ref), with the bounds derived there."""
import numpy as np
import pytest

import broadcast_gemm_amd as bga
import training_ref as ref
from gpu_util import log, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    bga.lib()


def T():
    from broadcast_gemm_amd import training
    return training


def dev(a, dtype=None):
    x = torch().from_numpy(np.ascontiguousarray(a))
    return (x if dtype is None else x.to(dtype)).cuda()


def f64(x):
    return x.detach().double().cpu().numpy()


def word():
    return torch().zeros(1, dtype=torch().int32, device="cuda")


def status(st):
    from broadcast_gemm_amd import history
    return history.kv_status(st)


def bf16(g, *shape, size=1.0):
    """Normal values that bf16 holds, as a tensor and in float64."""
    t = torch()
    x = t.from_numpy(g.normal(size=shape) * size).to(t.bfloat16)
    return x, x.double().numpy()


class Inputs:
    def __init__(self, seed, B_u, B_c, H_q, H_kv, L_q, L_kv, dim, ragged=True, causal=False, dropout=0.0, padding=0, empty_users=False, size=1.0, scale=0.0):
        g = np.random.default_rng(seed)
        self.q, self.Q = bf16(g, B_c, H_q, L_q, dim, size=size)
        self.k, self.K = bf16(g, B_u, H_kv, L_kv, dim, size=size)
        self.v, self.V = bf16(g, B_u, H_kv, L_kv, dim)
        self.do, self.dO = bf16(g, B_c, H_q, L_q, dim)
        self.mp = g.integers(0, max(1, B_u // 2) if empty_users else B_u, B_c).astype(np.int32)
        if padding:
            self.mp[g.permutation(B_c)[:padding]] = -1
        self.lens = g.integers(0, L_kv + 1, B_u).astype(np.int32) if ragged else None
        self.positions = g.integers(-1, L_kv + 3, (B_c, L_q)).astype(np.int32) if causal else None
        self.rng = (int(g.integers(0, 1 << 62)), int(g.integers(0, 1 << 32)))
        self.dropout, self.scale = dropout, scale

    def how(self, device=True):
        t = torch()
        d = dict(dropout=self.dropout, scale=self.scale, lens=self.lens, positions=self.positions, rng=self.rng)
        if device:
            for n in ("lens", "positions"):
                d[n] = None if d[n] is None else dev(d[n])
            d["rng"] = t.tensor(self.rng, dtype=t.int64, device="cuda")
        return d

    def want(self):
        return ref.attention(self.Q, self.K, self.V, self.mp, dO=self.dO, **self.how(False))

    def run(self, q=None, k=None, v=None, do=None, st=None, **kw):
        st = word() if st is None else st
        q, k, v, do = (b.cuda() if a is None else a for a, b in ((q, self.q), (k, self.k), (v, self.v), (do, self.do)))
        mp = dev(self.mp)
        O, lse = T().attention(q, k, v, mp, st, **self.how(), **kw)
        dQ, dK, dV = T().attention_backward(do, q, k, v, O, lse, mp, st, **self.how(), **kw)
        return dict(O=O, lse=lse, dQ=dQ, dK=dK, dV=dV)


def compare(got, want, what):
    for name in ("O", "lse", "dQ", "dK", "dV"):
        x, y = f64(got[name]), want[name]
        gone = np.isneginf(y)
        assert np.array_equal(gone, np.isneginf(x)) and np.isfinite(x[~gone]).all(), f"{what}: {name}"
        h = 0.0 if name == "lse" else ref.B8
        ok, share = ref.within(np.where(gone, 0, x), np.where(gone, 0, y), want["off"][name], h)
        log(f"  {what} {name}: {share:.2f} of the bound")
        assert ok, f"{what}: {name} outside, {share:.3g} of its bound"


SHAPES = [
    # B_u, B_c, H_q, H_kv, L_q, L_kv, dim
    (1, 1, 1, 1, 1, 1, 64), (1, 1, 1, 1, 1, 1, 128), (3, 7, 2, 1, 1, 64, 64), (2, 9, 2, 2, 3, 65, 128), (5, 40, 4, 2, 16, 130, 64), (4, 33, 3, 3, 33, 63, 128),
    (2, 65, 8, 2, 1, 257, 128), (7, 5, 1, 1, 64, 300, 64), (1, 300, 2, 1, 2, 96, 64), (30, 64, 6, 2, 1, 31, 128), (2, 3, 2, 2, 1, 4500, 64),
    (1, 2, 4, 1, 5, 2000, 128), (130, 257, 1, 1, 1, 20, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["whole", "ragged", "causal", "dropout"])
def test_attention_and_its_gradients(shape, kind):
    log(f"attention {shape} {kind}")
    x = Inputs(sum(shape), *shape, ragged=kind != "whole", causal=kind in ("causal", "dropout"), dropout=0.3 if kind == "dropout" else 0.0,
               padding=shape[1] // 5 if kind != "whole" else 0, empty_users=kind == "ragged")
    st = word()
    compare(x.run(st=st), x.want(), f"{shape} {kind}")
    assert status(st) == bga.IKBO_OK


@pytest.mark.parametrize("dropout", [1 / 256, 0.5, 255 / 256])
@pytest.mark.parametrize("dim", [64, 128])
def test_every_dropout_at_one_key_and_many(dropout, dim):
    for L_kv in (1, 70):
        x = Inputs(8, 2, 12, 2, 1, 3, L_kv, dim, ragged=False, dropout=dropout)
        log(f"dropout {dropout} dim={dim} L_kv={L_kv}")
        compare(x.run(), x.want(), f"dropout {dropout}")


@pytest.mark.parametrize("L_kv", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257])
def test_lengths_at_the_edges_of_tiles(L_kv):
    x = Inputs(L_kv, 3, 6, 2, 1, 5, L_kv, 64, dropout=0.25)
    x.lens = np.array([L_kv, max(0, L_kv - 1), 0], np.int32)
    log(f"edges L_kv={L_kv}")
    compare(x.run(), x.want(), f"L_kv {L_kv}")


@pytest.mark.parametrize("rows", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 513, 1100])
def test_rows_at_the_edges_of_tiles(rows):
    """One user with many rows beside one with a single row and one without."""
    x = Inputs(rows, 3, rows + 1, 1, 1, 1, 70, 128, ragged=False, causal=True)
    x.mp = np.where(np.arange(rows + 1) == rows // 2, 2, 0).astype(np.int32)
    log(f"edges rows={rows}")
    compare(x.run(), x.want(), f"rows {rows}")


def test_large_scores():
    """Scores of several hundred: one weight is 1 and the others vanish."""
    x = Inputs(5, 3, 20, 2, 1, 4, 200, 64, size=7.0)
    log("large scores")
    compare(x.run(), x.want(), "large scores")
    x = Inputs(6, 3, 20, 2, 1, 4, 200, 128, size=3.0, scale=1.5, dropout=0.1)
    compare(x.run(), x.want(), "a scale")


def test_many_users_and_candidates():
    """More users than threads of the grouping, and a map that names them in no order."""
    x = Inputs(4, 2000, 3001, 1, 1, 1, 9, 64, padding=50, empty_users=True)
    log("many users")
    compare(x.run(), x.want(), "many users")
    x = Inputs(5, 4096, 60, 1, 1, 1, 5, 64)
    compare(x.run(), x.want(), "most users")


@pytest.mark.parametrize("shape", [
    # B_u, B_c, H_q, H_kv, L_q, L_kv, dim: around the sizes where blocks find their own places, with and without cut keys
    (64, 1024, 1, 1, 4, 40, 64), (64, 1025, 1, 1, 1, 40, 64), (65, 1024, 1, 1, 1, 40, 64), (2, 1024, 4, 1, 1, 300, 64), (2, 1024, 4, 1, 1, 40, 128),
    (1, 512, 1, 1, 1, 600, 64), (1, 513, 1, 1, 1, 600, 64), (1, 128, 4, 1, 1, 30, 128), (16, 512, 4, 1, 1, 520, 64), (16, 511, 4, 1, 1, 520, 128),
    (16, 513, 4, 1, 1, 520, 128), (64, 1, 8, 1, 16, 1300, 128), (33, 1000, 2, 1, 1, 20, 64),
    # and of many candidates, whose grouping takes several turns, and many rows of a user
    (23, 9001, 1, 1, 2, 20, 64), (3, 2500, 2, 1, 1, 100, 128), (2, 1300, 2, 1, 2, 70, 64)])
@pytest.mark.parametrize("dropout", [0.0, 0.2])
def test_both_ways_of_grouping(shape, dropout):
    log(f"grouping {shape} dropout={dropout}")
    x = Inputs(sum(shape), *shape, causal=bool(dropout) or shape[1] % 2 == 1, dropout=dropout, padding=shape[1] // 7)
    if shape[1] > 8:
        x.mp[::9] = shape[0] // 2   # one user more often than the others
    st = word()
    got, again = x.run(st=st), x.run(st=st)
    assert status(st) == bga.IKBO_OK
    assert all(torch().equal(got[n], again[n]) for n in got)
    compare(got, x.want(), f"{shape}")


@pytest.mark.parametrize("shape", [(3, 700, 6, 2, 4, 30, 64), (70, 1500, 2, 1, 8, 20, 128), (2, 65, 64, 64, 40, 10, 64)])
def test_mostly_padding(shape):
    """Nine of ten candidates are padding: their rows are shared by many waves."""
    log(f"padding {shape}")
    x = Inputs(21, *shape, padding=shape[1] * 9 // 10)
    out = x.run()
    compare(out, x.want(), f"{shape}")
    assert not f64(out["O"])[x.mp < 0].any() and not f64(out["dQ"])[x.mp < 0].any()


@pytest.mark.parametrize("users", [9, 70])
@pytest.mark.parametrize("dim", [64, 128])
def test_keys_that_no_query_sees(users, dim):
    """Users without candidates, ranges of keys behind every position and behind histories stand between others: zeros, and
    nothing of the former is read."""
    x = Inputs(users + dim, users, 80, 2, 1, 2, 700, dim, causal=True, padding=5, empty_users=True)
    x.positions[:] = x.positions % 230
    x.lens[1] = 700
    k, v = x.k.cuda(), x.v.cuda()
    none = ~np.isin(np.arange(users), x.mp)
    k[none], v[none] = float("nan"), float("inf")
    log(f"keys without rows: {users} users, head {dim}")
    got = x.run(k=k, v=v)
    compare(got, x.want(), f"{users} users, head {dim}")
    for n in ("dK", "dV"):
        assert none.sum() > 3 and not f64(got[n])[none].any() and not f64(got[n])[:, :, 230:].any()


def test_strided_tensors():
    """Queries and gradients with tokens before heads, K and V out of one projection, K shared by all users, an
    expanded upstream gradient."""
    t = torch()
    x = Inputs(9, 3, 10, 4, 2, 6, 100, 64, causal=True)
    log("strides")
    want = x.want()
    q = x.q.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    do = x.do.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    kv = t.stack([x.k, x.v], 3).cuda()                       # [B_u, H, L, 2, dim]
    k, v = kv[:, :, :, 0], kv[:, :, :, 1]
    assert not q.is_contiguous() and k.stride(2) == 128
    compare(x.run(q=q, k=k, v=v, do=do), want, "strides")
    x.K[:], x.dO[:] = x.K[:1], x.dO[:, :, :1]
    k = k[:1].expand(3, -1, -1, -1)
    do = do[:, :, :1].expand(-1, -1, 6, -1)
    compare(x.run(k=k, v=v, do=do), x.want(), "expanded")


def test_wide_offsets():
    """Users and candidates more than 2^32 bytes apart."""
    t = torch()
    x = Inputs(10, 3, 4, 1, 1, 2, 70, 64)
    x.mp = np.array([2, 0, 1, 2], np.int32)
    log("wide offsets")
    step = (1 << 31) + 4096                                  # elements: 4.3 GB
    big = t.empty(3 * step + 2 * 4 * 64, dtype=t.bfloat16, device="cuda")

    def far(y):
        z = big.as_strided((y.shape[0], 1, y.shape[2], 64), (step if y.shape[0] == 3 else step * 3 // 4, 64 * y.shape[2], 64, 1))
        return z.copy_(y.cuda())

    want = x.want()
    compare(x.run(k=far(x.k)), want, "far keys")
    compare(x.run(q=far(x.q)), want, "far queries")
    compare(x.run(do=far(x.do)), want, "far gradients")


def test_rows_of_one_user_whose_notes_pass_2_to_31_bytes():
    """45 million candidates of one user, each of which sees the first of 50000 tokens: one chunk of rows, 48 bytes of notes each.
    O is that token's V and the weights are 1, so dV is the sum of dO there, and dQ and dK are zero."""
    t = torch()
    n, dim = 45_000_000, 64
    log("45 million rows")
    bf = dict(dtype=t.bfloat16, device="cuda")
    k, v = t.randn(1, 1, 50_000, dim, **bf), t.randn(1, 1, 50_000, dim, **bf)
    q = t.randn(1, 1, 1, dim, **bf).expand(n, -1, -1, -1)
    lse = (q[0, 0, 0].double() @ k[0, 0, 0].double() / 8).float().expand(n, 1, 1).contiguous()
    do = t.zeros(n, 1, 1, dim, **bf)
    far = [0, 1, n // 2, 43_000_000, 44_739_264, n - 65, n - 2, n - 1]    # 2^31 bytes of notes end with row 44739242
    do[far] = t.randn(len(far), 1, 1, dim, **bf)
    mp, positions, st = t.zeros(n, dtype=t.int32, device="cuda"), t.zeros(n, 1, dtype=t.int32, device="cuda"), word()
    dQ, dK, dV = T().attention_backward(do, q, k, v, v[:, :, :1].expand(n, -1, -1, -1), lse, mp, st, positions=positions)
    t.cuda.synchronize()
    assert status(st) == bga.IKBO_OK
    rows, size = f64(do[far]).reshape(len(far), dim), np.abs(f64(v[0, 0, 0]))
    # A score is a float32 sum of dim products, and so is the lse given: each weight is off by their rounding, and by half a step of bf16.
    w = 2 * (dim + 4) * ref.U24 * float((q[0, 0, 0].double() * k[0, 0, 0].double()).abs().sum()) / 8 + 2.0 ** -20
    want, off = rows.sum(0), np.abs(rows).sum(0) * (ref.B8 + w)
    assert (np.abs(f64(dV[0, 0, 0]) - want) <= off + ref.B8 * (np.abs(want) + off)).all()
    assert not dV[0, 0, 1:].any()
    # dS = P (dP - D), where D is the row's one P dP: off by P's error and twice that of dP, a float32 sum of dim products.
    ds = (np.abs(rows) @ size) * (2 * w + 2 * (dim + 4) * ref.U24)
    assert (np.abs(f64(dK[0, 0, 0])) <= ds.sum() / 8 * np.abs(f64(q[0, 0, 0])) * 1.01 + 1e-30).all() and not dK[0, 0, 1:].any()
    assert float(dQ[far].abs().max()) <= ds.max() / 8 * float(k[0, 0, 0].abs().max()) * 1.01
    assert not dQ[500::1000].any()


def test_what_is_masked_is_not_read():
    """NaN and infinity behind the histories, in the rows of padding and in the gradients of queries that see nothing."""
    t = torch()
    x = Inputs(11, 4, 20, 2, 1, 3, 90, 64, causal=True, padding=4, dropout=0.2)
    x.lens[0] = 0
    x.mp[:3] = 0, 1, 1
    x.positions[1, 0] = -1
    want = x.want()
    k, v, q, do = x.k.cuda(), x.v.cuda(), x.q.cuda(), x.do.cuda()
    for u, n in enumerate(x.lens):
        k[u, :, n:] = float("nan")
        v[u, :, n:] = float("inf")
    for b, u in enumerate(x.mp):
        for l in range(3):
            if u < 0 or x.lens[u] == 0 or x.positions[b, l] < 0:
                q[b, :, l], do[b, :, l] = float("nan"), float("inf")
    log("masked places")
    compare(x.run(q=q, k=k, v=v, do=do), want, "masked")


def test_nonfinite_values_reach_their_own_rows_only():
    t = torch()
    x = Inputs(12, 2, 8, 2, 2, 4, 50, 64, ragged=False)
    x.mp = (np.arange(8) % 2).astype(np.int32)
    v, q = x.v.cuda(), x.q.cuda()
    v[0, 0, 7, 3] = float("nan")
    q[5, 1, 2, 0] = float("nan")
    log("nonfinite")
    got, want = x.run(q=q, v=v), x.want()
    O = f64(got["O"])
    bad = np.isnan(O)
    assert bad[0::2, 0, :, 3].all() and bad[5, 1, 2].all()
    bad[0::2, 0, :, 3] = False
    bad[5, 1, 2] = False
    assert not bad.any()
    assert np.isfinite(f64(got["dK"])[0, 1]).all() and np.isfinite(f64(got["dV"])[1, 0]).all() and np.isnan(f64(got["dK"])[1, 1]).any()
    assert np.isfinite(f64(got["dQ"])[1::2, 0]).all()


def test_conditions_are_recorded():
    t = torch()
    x = Inputs(13, 3, 9, 2, 1, 2, 40, 64)
    x.mp[:] = np.arange(9) % 3
    want = {}
    st = word()
    x.lens[:] = 100, -3, 20
    got = x.run(st=st)
    assert status(st) == bga.IKBO_ERR_PAGE_RANGE and status(st) == bga.IKBO_OK
    x.lens[:] = 40, 0, 20
    compare(got, x.want(), "clamped lengths")
    x.mp[2], x.mp[5] = 3, -7
    got = x.run(st=st)
    assert status(st) == bga.IKBO_ERR_MAP_RANGE
    x.mp[[2, 5]] = -1
    compare(got, x.want(), "map out of range")


def test_conditions_of_many_candidates_are_recorded():
    """As above, where the grouping is a launch of its own."""
    x = Inputs(13, 70, 99, 2, 1, 2, 40, 64)
    st = word()
    x.lens[:] = 20
    x.lens[69] = -1
    got = x.run(st=st)
    assert status(st) == bga.IKBO_ERR_PAGE_RANGE and status(st) == bga.IKBO_OK
    x.lens[69] = 0
    compare(got, x.want(), "clamped lengths")
    x.mp[98] = 70
    got = x.run(st=st)
    assert status(st) == bga.IKBO_ERR_MAP_RANGE
    x.mp[98] = -1
    compare(got, x.want(), "map out of range")


def test_no_candidates_and_padding_alone():
    t = torch()
    x = Inputs(14, 2, 3, 2, 1, 2, 40, 64)
    q = t.empty(0, 2, 2, 64, dtype=t.bfloat16, device="cuda")
    none = t.empty(0, dtype=t.int32, device="cuda")
    k, v = x.k.cuda(), x.v.cuda()
    O, lse = T().attention(q, k, v, none, word())
    assert O.shape == q.shape and lse.shape == (0, 2, 2)
    dQ, dK, dV = T().attention_backward(q, q, k, v, O, lse, none, word())
    assert dQ.shape == q.shape and not dK.any() and not dV.any()
    x.mp[:] = -1
    compare(x.run(), x.want(), "padding alone")


def test_same_call_same_bits_and_other_numbers():
    t = torch()
    x = Inputs(15, 5, 120, 8, 2, 3, 700, 64, causal=True, dropout=0.4)
    a, b = x.run(), x.run()
    assert all(t.equal(a[n], b[n]) for n in a)
    x.rng = (x.rng[0], x.rng[1] + (1 << 32))
    assert t.equal(x.run()["O"], a["O"])                     # offsets count modulo 2^32
    x.rng = (x.rng[0], x.rng[1] + 1)
    c = x.run()
    assert not t.equal(c["O"], a["O"]) and t.equal(c["lse"], a["lse"])


def test_streams_and_replayed_graphs():
    """Two captured steps that share nothing but their inputs, replayed between eager work on two streams, with other
    numbers and lengths for every replay."""
    t = torch()
    xs = [Inputs(16, 4, 50, 4, 2, 3, 200, 64, dropout=0.2), Inputs(17, 2, 31, 2, 2, 2, 900, 128, causal=True, dropout=0.1),
          Inputs(18, 70, 300, 2, 2, 2, 300, 64, dropout=0.1)]
    steps = []
    for x in xs:
        st, mp, how = word(), dev(x.mp), x.how()
        ten = [y.cuda() for y in (x.q, x.k, x.v, x.do)]

        def step(ten=ten, mp=mp, st=st, how=how):
            O, lse = T().attention(*ten[:3], mp, st, **how)
            return O, lse, *T().attention_backward(ten[3], *ten[:3], O, lse, mp, st, **how)
        steps.append((step, how))
    side = t.cuda.Stream()
    t.cuda.synchronize()
    with t.cuda.stream(side):
        for step, _ in steps:
            step()
    t.cuda.synchronize()
    graphs = []
    for step, how in steps:
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for turn in range(4):
        for step, how in steps:
            how["rng"][1] += 1
            how["lens"] += (-1 if turn % 2 else 1) * (how["lens"] > 5)
        t.cuda.synchronize()
        with t.cuda.stream(side):
            eager = [step() for step, _ in steps]
        for g, _ in graphs:
            g.replay()
        t.cuda.synchronize()
        for (_, out), want in zip(graphs, eager):
            assert all(t.equal(a, b) for a, b in zip(out, want)), turn
    step, how = steps[0]
    handle = side.cuda_stream
    x = xs[0]
    O, lse = T().attention(x.q.cuda(), x.k.cuda(), x.v.cuda(), dev(x.mp), word(), stream=handle, **how)
    t.cuda.synchronize()
    assert t.equal(O, eager[0][0]) and t.equal(lse, eager[0][1])


def test_refusals_of_the_binding():
    t = torch()
    x = Inputs(18, 2, 4, 2, 1, 3, 40, 64, dropout=0.5)
    q, k, v, mp, st, how = x.q.cuda(), x.k.cuda(), x.v.cuda(), dev(x.mp), word(), x.how()
    bad = [(q.float(), k, v, mp, st), (q, k.float(), v, mp, st), (q[0], k, v, mp, st), (q.transpose(2, 3), k, v, mp, st), (q, k, v, mp.long(), st),
           (q, k, v.cpu(), mp, st), (q, k, v, mp, st.long()), (q, k, v, mp.cpu(), st)]
    for args in bad:
        with pytest.raises(ValueError):
            T().attention(*args, **how)
    for change in (dict(rng=None), dict(rng=how["rng"].int()), dict(rng=how["rng"][:1]), dict(lens=how["lens"].long())):
        with pytest.raises(ValueError):
            T().attention(q, k, v, mp, st, **{**how, **change})
    for args in ((q, k, v[:1], mp, st), (q, k, v, mp[:3], st), (q[..., :32], k[..., :32], v[..., :32], mp, st), (q[:, :, :, :], k[:, :, :0], v[:, :, :0], mp, st)):
        with pytest.raises(bga.IkboError):
            T().attention(*args, **how)
    for change in (dict(lens=how["lens"][:1]), dict(dropout=1.0), dict(dropout=0.0001), dict(scale=-1.0), dict(positions=dev(np.zeros((4, 2), np.int32)))):
        with pytest.raises(bga.IkboError):
            T().attention(q, k, v, mp, st, **{**how, **change})
    odd = t.empty(q.numel() + 8, dtype=q.dtype, device="cuda")[4:4 + q.numel()].view(q.shape)
    with pytest.raises(bga.IkboError) as e:
        T().attention(odd, k, v, mp, st, **how)
    assert e.value.status == bga.IKBO_ERR_ALIGNMENT
    O, lse = T().attention(q, k, v, mp, st, **how)
    with pytest.raises(bga.IkboError):
        T().attention_backward(O[:3], q, k, v, O, lse, mp, st, **how)
    with pytest.raises(ValueError):
        T().attention_backward(O, q, k, v, O, lse.double(), mp, st, **how)
    with pytest.raises(ValueError):
        T().attention_backward(O.float(), q, k, v, O, lse, mp, st, **how)


# ---- dropout -------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 2047, 2048, 2049, 70001])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(dtype, n, residual):
    t = torch()
    g = np.random.default_rng(n)
    dtype = getattr(t, dtype)
    x, r = (t.from_numpy(g.normal(size=n)).to(dtype) for _ in range(2))
    h = t.finfo(dtype).eps / 2
    for p in (0.0, 1 / 65536, 0.1, 0.9, 65535 / 65536):
        rng = (int(g.integers(0, 1 << 62)), int(g.integers(0, 1 << 32)))
        log(f"dropout {dtype} n={n} residual={residual} p={p}")
        y = f64(T().dropout(x.cuda(), p, t.tensor(rng, device="cuda"), residual=r.cuda() if residual else None))
        kept = np.where(ref.elements_kept(n, p, rng), f64(x) / (1 - round(65536 * p) / 65536), 0.0)
        want = kept + (f64(r) if residual else 0.0)
        # The factor, the product and the sum round in float32, and then the type.
        off = 2 * ref.U24 * np.abs(kept) + ref.U24 * np.abs(want)
        assert (np.abs(y - want) <= off * (1 + h) + h * np.abs(want)).all()
        if not residual:
            assert (y[kept == 0] == 0).all()


def test_dropout_places():
    """In place, over the residual, at odd addresses, with NaN and infinity in what goes."""
    t = torch()
    rng = t.tensor([3, 4], device="cuda")
    g = t.Generator(device="cuda").manual_seed(1)
    for dtype in (t.bfloat16, t.float32):
        base = t.randn(5001, generator=g, device="cuda").to(dtype)
        want = T().dropout(base, 0.3, rng)
        add = t.randn(5001, generator=g, device="cuda").to(dtype)
        both = T().dropout(base, 0.3, rng, residual=add)
        room = t.empty(5010, dtype=dtype, device="cuda")
        for at in (0, 1, 3, 8):
            x = room[at:at + 5001]
            x.copy_(base)
            assert t.equal(T().dropout(x, 0.3, rng), want)
            assert T().dropout(x, 0.3, rng, out=x) is x and t.equal(x, want)
            x.copy_(add)
            assert t.equal(T().dropout(base, 0.3, rng, residual=x, out=x), both)
        kept = t.from_numpy(ref.elements_kept(5001, 0.3, (3, 4))).cuda()
        x = t.where(kept, base, float("nan"))
        x[~kept & (t.arange(5001, device="cuda") % 2 == 0)] = float("inf")
        assert t.equal(T().dropout(x, 0.3, rng), want) and t.equal(T().dropout(x, 0.3, rng, residual=add), both)
        with pytest.raises(ValueError):
            T().dropout(room[:5000], 0.3, rng, out=room[1:5001])
        with pytest.raises(ValueError):
            T().dropout(base, 0.3, rng, residual=room[:5001], out=room[2:5003])
        with pytest.raises(ValueError):
            T().dropout(room[:5000].view(100, 50).t(), 0.3, rng)
        with pytest.raises(ValueError):
            T().dropout(base, 0.3, rng.int())
        with pytest.raises(ValueError):
            T().dropout(base, 0.3, rng, residual=add[:100])
        with pytest.raises(bga.IkboError):
            T().dropout(base, 1.0, rng)
    with pytest.raises(ValueError):
        T().dropout(t.zeros(8, dtype=t.float16, device="cuda"), 0.3, rng)
    assert T().dropout(t.empty(0, device="cuda"), 0.3, rng).numel() == 0


def test_dropout_of_more_than_2_to_32_elements():
    """The last elements take the counters behind 2^29, whose generator words and places pass 32 bits."""
    t = torch()
    n = (1 << 32) + 77
    x = t.ones(n, dtype=t.bfloat16, device="cuda")
    rng = t.tensor([11, 12], device="cuda")
    log("dropout of 2^32 elements")
    y = T().dropout(x, 0.5, rng, out=x)[-4096 - 77:].cpu()
    counter = np.zeros((-(-(4096 + 77) // 8), 4), np.uint64)
    at = (1 << 32) - 4096
    counter[:, 0] = at // 8 + np.arange(len(counter))
    counter[:, 2], counter[:, 3] = 0xFFFFFFFF, 12
    words = ref.philox(counter, 11)
    kept = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], -1).reshape(-1)[:4096 + 77] >= 32768
    assert np.array_equal(f64(y), np.where(kept, 2.0, 0.0))


# ---- together ------------------------------------------------------------------------------


def test_modules_run_together():
    """Rotary positions, attention with dropout, dropout onto the residual stream, the LCE with dropout: a step's gradients
    are those of the same calls made by hand, and evaluation drops nothing."""
    t = torch()
    from broadcast_gemm_amd.autograd import IkboAttention, IkboDropout, IkboLce, IkboRope
    from broadcast_gemm_amd import history
    x = Inputs(20, 3, 12, 4, 2, 8, 60, 64, causal=True, padding=2)
    attend, drop = IkboAttention(dropout=0.2, seed=5).cuda(), IkboDropout(0.25, seed=6).cuda()
    rope, lce = IkboRope(64).cuda(), IkboLce(10, 32, 8, 64, dropout=0.1).cuda()
    q, k, v = (y.cuda().requires_grad_() for y in (x.q, x.k, x.v))
    mp, lens, positions = dev(x.mp).long(), dev(x.lens), dev(np.maximum(x.positions, 0))
    U = t.randn(3, 10, 64, device="cuda").to(t.bfloat16)

    def forward():
        flat = q.transpose(1, 2).reshape(-1, 4, 64)
        turned = rope(flat, None, positions.reshape(-1))[0].view(12, 8, 4, 64).transpose(1, 2)
        O = attend(turned, k, v, mp, lens=lens, positions=positions)
        return turned, O, drop(O, q)

    turned, O, y = forward()
    Y = lce(U, y.reshape(12, 32, 64), mp.clamp(min=0))
    dy = t.randn_like(y.float()).to(t.bfloat16)
    log("together")
    t.autograd.backward([y, Y], [dy, t.zeros_like(Y)])
    t.cuda.synchronize()
    assert attend.check() == bga.IKBO_OK
    i32 = [z.to(t.int32) for z in (mp, lens, positions)]
    st = word()
    how = dict(lens=i32[1], positions=i32[2], dropout=0.2, rng=t.tensor([5, 0], device="cuda"))
    O2, lse = T().attention(turned.detach(), k.detach(), v.detach(), i32[0], st, **how)
    assert t.equal(O, O2) and t.equal(y, T().dropout(O2, 0.25, t.tensor([6, 0], device="cuda"), residual=q.detach()))
    dO = T().dropout(dy, 0.25, t.tensor([6, 0], device="cuda"))
    dt, dk, dv = T().attention_backward(dO, turned.detach(), k.detach(), v.detach(), O2, lse, i32[0], st, **how)
    assert t.equal(k.grad, dk) and t.equal(v.grad, dv)
    back = history.rope(dt.transpose(1, 2).reshape(-1, 4, 64), None, i32[2].reshape(-1), rope.freq, inverse=True)[0]
    assert t.equal(q.grad, back.view(12, 8, 4, 64).transpose(1, 2) + dy)
    assert attend.rng.tolist() == [5, 1] and drop.rng.tolist() == [6, 1]
    assert abs(float((Y == 0).float().mean()) - 0.1) < 0.05
    for m in (attend, drop, lce):
        m.eval()
    a, b = forward()[1:], forward()[1:]
    assert t.equal(a[0], b[0]) and t.equal(a[1], b[1]) and attend.rng.tolist() == [5, 1]
    lce._plans.close()


def test_module_takes_any_strides_and_only_what_needs_gradients():
    t = torch()
    from broadcast_gemm_amd.autograd import IkboAttention
    x = Inputs(21, 2, 5, 2, 2, 3, 40, 64, ragged=False)
    attend = IkboAttention().cuda()
    k, v = x.k.cuda(), x.v.cuda()
    q = x.q.transpose(2, 3).contiguous().cuda().transpose(2, 3).requires_grad_()   # elements of a row far apart
    O = attend(q, k, v, dev(x.mp))
    O.sum().backward()                                                             # an upstream gradient without strides
    x.dO[:] = 1.0
    want = x.want()
    ok, share = ref.within(f64(q.grad), want["dQ"], want["off"]["dQ"], ref.B8)
    assert ok, share
    ok, share = ref.within(f64(O), want["O"], want["off"]["O"], ref.B8)
    assert ok, share


def test_a_captured_training_step_draws_new_numbers():
    t = torch()
    from broadcast_gemm_amd.autograd import IkboAttention
    x = Inputs(22, 3, 20, 2, 1, 2, 100, 64)
    attend = IkboAttention(dropout=0.3, seed=9).cuda()
    q, k, v = (y.cuda().requires_grad_() for y in (x.q, x.k, x.v))
    mp, lens, do = dev(x.mp), dev(x.lens), x.do.cuda()
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        O = attend(q, k, v, mp, lens=lens)
        t.autograd.grad(O, (q, k, v), do)
    t.cuda.current_stream().wait_stream(side)
    del O
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        O = attend(q, k, v, mp, lens=lens)
        grads = t.autograd.grad(O, (q, k, v), do)
    seen = []
    for turn in range(3):
        offset = int(attend.rng[1])
        g.replay()
        t.cuda.synchronize()
        assert int(attend.rng[1]) == offset + 1
        how = dict(lens=lens, dropout=0.3, rng=t.tensor([9, offset], device="cuda"))
        O2, lse = T().attention(q.detach(), k.detach(), v.detach(), mp, word(), **how)
        want = T().attention_backward(do, q.detach(), k.detach(), v.detach(), O2, lse, mp, word(), **how)
        assert t.equal(O, O2) and all(t.equal(a, b) for a, b in zip(grads, want))
        seen.append(O.clone())
    assert not t.equal(seen[0], seen[1]) and not t.equal(seen[1], seen[2])


@pytest.mark.parametrize("reentrant", [False, True])
def test_gradients_under_activation_checkpointing(reentrant):
    """Two layers of attention, dropout and the LCE, whose forward runs again in the backward: the same outputs and gradients as without,
    from the same state of torch's generator."""
    t = torch()
    from torch.utils.checkpoint import checkpoint
    from broadcast_gemm_amd.autograd import IkboAttention, IkboDropout, IkboLce
    x = Inputs(23, 3, 12, 4, 2, 8, 60, 64, padding=2)
    attend, drop, lce = IkboAttention(dropout=0.2).cuda(), IkboDropout(0.25).cuda(), IkboLce(10, 32, 32, 64, dropout=0.1).cuda()
    mp, lens = dev(x.mp), dev(x.lens)
    users = mp.clamp(min=0)
    U, dY = t.randn(3, 10, 64, device="cuda").to(t.bfloat16), x.do.cuda()
    log(f"checkpointing, reentrant={reentrant}")

    def layer(q, k, v):
        y = drop(attend(q, k, v, mp, lens=lens), q)
        return lce(U, y.reshape(12, 32, 64), users).view(12, 4, 8, 64)

    def step(call):
        t.manual_seed(31)
        leaves = [y.cuda().requires_grad_() for y in (x.q, x.k, x.v)]
        lce.W_u.grad = lce.W_c.grad = None
        Y = call(call(*leaves), *leaves[1:])
        Y.backward(dY)
        return [Y.detach()] + [y.grad for y in leaves + [lce.W_u, lce.W_c]]

    want = step(layer)
    got = step(lambda *a: checkpoint(layer, *a, use_reentrant=reentrant))
    t.cuda.synchronize()
    assert attend.check() == bga.IKBO_OK
    assert all(t.equal(a, b) for a, b in zip(got, want))
    assert not t.equal(layer(*(y.cuda() for y in (x.q, x.k, x.v))), layer(*(y.cuda() for y in (x.q, x.k, x.v))))
    lce._plans.close()


@pytest.mark.parametrize("shape", [(3, 12, 10, 32, 8, 64), (15, 200, 40, 64, 96, 160), (1, 1, 8, 8, 5, 128)])
def test_lce_with_dropout(shape):
    """Output and gradients are those of the LCE without dropout and of the dropout, one behind the other, with the same numbers."""
    t = torch()
    from broadcast_gemm_amd.autograd import IkboLce
    B_u, B_c, K_u, K_c, M, D = shape
    g = t.Generator(device="cuda").manual_seed(3)
    U, C, dY = (t.randn(*s, generator=g, device="cuda").to(t.bfloat16) for s in ((B_u, K_u, D), (B_c, K_c, D), (B_c, M, D)))
    mp = t.randint(0, B_u, (B_c,), generator=g, device="cuda")
    lce = IkboLce(K_u, K_c, M, D, dropout=0.1).cuda()
    log(f"LCE with dropout {shape}")

    def step(dY):
        for y in (U, C, lce.W_u, lce.W_c):
            y.grad = None
            y.requires_grad_()
        Y = lce(U, C, mp)
        Y.backward(dY)
        return Y.detach(), [y.grad for y in (U, C, lce.W_u, lce.W_c)]

    t.manual_seed(17)
    Y, grads = step(dY)
    t.manual_seed(17)
    rng = t.randint(0, 1 << 62, (2,), device="cuda")         # what the call took
    lce.eval()
    plain, want = step(T().dropout(dY, 0.1, rng))
    kept = ref.elements_kept(Y.numel(), 0.1, rng.tolist()).reshape(Y.shape)
    assert 0 < kept.mean() < 1 and not f64(Y)[~kept].any()
    # The factor and the product round in float32, and then bf16 does.
    exact = np.where(kept, f64(plain) / (1 - round(65536 * 0.1) / 65536), 0.0)
    assert (np.abs(f64(Y) - exact) <= np.abs(exact) * (ref.B8 + 3 * ref.U24)).all()
    assert all(t.equal(a, b) and a.any() for a, b in zip(grads, want))
    lce._plans.close()


@pytest.mark.parametrize("kind", ["row", "float32", "wider", "number"])
def test_residuals_that_are_not_like_the_activations(kind):
    """What evaluation adds, training adds too: of another shape or type, with gradients in the residual's shape."""
    t = torch()
    from broadcast_gemm_amd.autograd import IkboDropout
    g = t.Generator(device="cuda").manual_seed(2)
    x = t.randn(6, 35, generator=g, device="cuda").to(t.bfloat16).requires_grad_()
    shape = dict(row=(35,), float32=(6, 35), wider=(3, 6, 35), number=())[kind]
    r = t.randn(shape, generator=g, device="cuda").to(t.float32 if kind == "float32" else t.bfloat16).requires_grad_()
    r = 0.5 if kind == "number" else r
    drop = IkboDropout(0.25, seed=4).cuda()
    log(f"residual {kind}")
    y = drop(x, r)
    kept = T().dropout(x.detach(), 0.25, t.tensor([4, 0], device="cuda"))
    assert t.equal(y, r + kept)
    dy = t.randn(y.shape, generator=g, device="cuda").to(y.dtype)
    y.backward(dy)
    dx = dy.sum(0) if kind == "wider" else dy.to(x.dtype)
    assert t.equal(x.grad, T().dropout(dx, 0.25, t.tensor([4, 0], device="cuda")))
    if kind != "number":
        assert t.equal(r.grad, dy.sum(0) if kind == "row" else dy)
    z = drop.eval()(x, r)
    assert z.shape == y.shape and z.dtype == y.dtype


def test_module_with_numbers_beyond_32_bits():
    """Positions without a bound, and users and lengths that 32 bits would wrap into others, are what they are."""
    t = torch()
    from broadcast_gemm_amd.autograd import IkboAttention
    x = Inputs(24, 3, 10, 2, 1, 2, 50, 64)
    x.lens[:] = 50, 20, 50
    attend, q, k, v = IkboAttention().cuda(), x.q.cuda(), x.k.cuda(), x.v.cuda()
    mp, lens = dev(x.mp).long(), dev(x.lens).long()
    log("64-bit numbers")
    want = attend(q, k, v, mp, lens=lens)
    assert attend.check() == bga.IKBO_OK
    last = t.iinfo(t.int64).max
    assert t.equal(attend(q, k, v, mp, lens=lens, positions=t.full((10, 2), last, device="cuda")), want)
    assert not attend(q, k, v, mp, lens=lens, positions=t.full((10, 2), -last, device="cuda")).any()
    assert attend.check() == bga.IKBO_OK
    far = mp.clone()
    far[3] += 1 << 32
    got = attend(q, k, v, far, lens=lens)
    assert attend.check() == bga.IKBO_ERR_MAP_RANGE and not got[3].any() and t.equal(got[:3], want[:3]) and t.equal(got[4:], want[4:])
    lens[0] += 1 << 32
    assert t.equal(attend(q, k, v, mp, lens=lens), want) and attend.check() == bga.IKBO_ERR_PAGE_RANGE


def test_a_replica_on_another_device_than_its_original():
    """As torch.nn.DataParallel makes them: a status word that has not followed is copied; a module that was never moved is refused."""
    from broadcast_gemm_amd.autograd import IkboAttention
    x = Inputs(25, 2, 5, 2, 1, 2, 40, 64, ragged=False)
    here, there = IkboAttention().cuda(), IkboAttention()
    args = x.q.cuda(), x.k.cuda(), x.v.cuda(), dev(x.mp)
    assert torch().equal(there._replicate_for_data_parallel()(*args), here(*args))
    with pytest.raises(ValueError):
        there(*args)


def test_a_captured_step_takes_numbers_from_torch():
    """Every replay has another mask, and its gradient the same mask as its output."""
    t = torch()
    from broadcast_gemm_amd.autograd import IkboDropout
    drop = IkboDropout(0.5).cuda()
    x, dy = t.ones(4099, device="cuda").requires_grad_(), t.full((4099,), 3.0, device="cuda")
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        t.autograd.grad(drop(x), x, dy)
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        y = drop(x)
        dx, = t.autograd.grad(y, x, dy)
    seen = []
    for _ in range(4):
        g.replay()
        t.cuda.synchronize()
        assert set(y.unique().tolist()) == {0.0, 2.0} and t.equal(dx, 3 * y)
        seen.append(y.detach().clone())
        seen.append(drop(x).detach())   # eager calls between the replays
    assert all(not t.equal(a, b) for i, a in enumerate(seen) for b in seen[:i])
