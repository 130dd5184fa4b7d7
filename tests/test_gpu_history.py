"""The cached-history operators on the GPU against their plain 64-bit forms (history_ref), with bounds derived there."""
import numpy as np
import pytest

import broadcast_gemm_amd as bga
import history_ref as ref
from gpu_util import log, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    bga.lib()


def H():
    from broadcast_gemm_amd import history
    return history


def dev(a, dtype=None):
    t = torch()
    x = t.from_numpy(np.ascontiguousarray(a))
    return (x if dtype is None else x.to(dtype)).cuda()


def f64(x):
    return x.detach().double().cpu().numpy()


def word():
    return torch().zeros(1, dtype=torch().int32, device="cuda")


def bounded(got, want, bound, dtype, what):
    """|got - want| within the bound and one rounding to the type."""
    h = ref.half_step(dtype)
    off = np.abs(got - want) - (bound * (1 + h) + h * np.abs(want) + 1e-37)
    assert np.isfinite(got).all(), what
    assert (off <= 0).all(), f"{what}: {(off > 0).sum()} of {off.size} values outside, by up to {off.max():.3g}"


# ---- page tables ---------------------------------------------------------------------------


def make_step(rng, B, width, P, free_extra, most, leave=0.2, zero=0.2):
    lens = rng.integers(0, width * P - most + 1, B)
    lens[rng.random(B) < zero] = 0
    counts = rng.integers(0, most + 1, B)
    counts[rng.random(B) < leave] = -1
    held = (-(-lens // P)).sum()
    need = (-(-(lens + np.maximum(counts, 0)) // P)).sum() - held
    N = int(held + need + free_extra)
    order = rng.permutation(N)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for i in range(B):
        k = -(-lens[i] // P)
        table[i, :k] = order[at:at + k]
        at += k
    ring = np.full(N, -1, np.int32)
    head = int(rng.integers(0, N))
    ring[(head + np.arange(N - held)) % N] = order[held:]
    return counts.astype(np.int32), lens.astype(np.int32), table, ring, head, int(N - held)


def run_tables(step, capacity, P, in_place=False):
    counts, lens, table, ring, head, free = step
    t = torch()
    state = t.tensor([head, free, 0, 0], dtype=t.int32, device="cuda")
    d = [dev(x) for x in (counts, lens, table, ring)]
    st = word()
    got = H().kv_tables(d[0], d[1], d[2], d[3], state, capacity, st, page_size=P, in_place=in_place)
    return got, d, state, H().kv_status(st)


@pytest.mark.parametrize("B, width, P, most, spare", [
    (1, 1, 1, 1, 1), (1, 3, 64, 100, 0), (5, 4, 64, 70, 9), (59, 9, 64, 1, 3), (64, 5, 7, 20, 100), (1023, 4, 16, 33, 17),
    (1025, 3, 64, 64, 0), (4096, 3, 64, 5, 1000), (300, 40, 64, 2000, 5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables(B, width, P, most, spare, in_place):
    rng = np.random.default_rng(B + most)
    step = make_step(rng, B, width, P, 3, most)
    capacity = int(np.maximum(step[0], 0).sum()) + spare
    log(f"tables B={B} width={width} P={P} most={most} in_place={in_place}")
    got, d, state, st = run_tables(step, capacity, P, in_place)
    table, ring = step[2].copy(), step[3].copy()
    want = ref.tables(step[0], step[1], table, ring, step[4], step[5], capacity, P)
    assert st == bga.IKBO_OK
    for name, x, y in zip(("slots", "positions", "rows", "starts", "lens"), got[:5], want[:5]):
        assert np.array_equal(x.cpu().numpy(), y), name
    assert got.state.tolist()[:3] == [want[5], want[6], 0]
    assert np.array_equal(d[2].cpu().numpy(), table) and np.array_equal(d[3].cpu().numpy(), ring)
    if in_place:
        assert np.array_equal(d[1].cpu().numpy(), want[4]) and state.tolist()[:3] == [want[5], want[6], 0]
    else:
        assert np.array_equal(d[1].cpu().numpy(), step[1]) and state.tolist() == [step[4], step[5], 0, 0]


@pytest.mark.parametrize("what, status", [
    ("pages", bga.IKBO_ERR_NO_PAGES), ("rows", bga.IKBO_ERR_NO_PAGES), ("columns", bga.IKBO_ERR_NO_PAGES),
    ("negative length", bga.IKBO_ERR_PAGE_RANGE), ("long length", bga.IKBO_ERR_PAGE_RANGE), ("count", bga.IKBO_ERR_PAGE_RANGE),
    ("head", bga.IKBO_ERR_PAGE_RANGE), ("free", bga.IKBO_ERR_PAGE_RANGE), ("huge counts", bga.IKBO_ERR_NO_PAGES)])
def test_tables_refuse_a_step_as_a_whole(what, status):
    rng = np.random.default_rng(5)
    counts, lens, table, ring, head, free = make_step(rng, 70, 6, 64, 0, 130, leave=0.1)
    capacity = int(np.maximum(counts, 0).sum()) + 4
    if what == "pages":
        free -= 1
    if what == "rows":
        capacity = int(np.maximum(counts, 0).sum()) - 1
    if what == "columns":
        lens[3], counts[3] = 6 * 64 - 4, 5
    if what == "negative length":
        lens[3], counts[3] = -1, 5
    if what == "long length":
        lens[3], counts[3] = 6 * 64 + 1, 0
    if what == "count":
        counts[3] = -2
    if what == "head":
        head = len(ring)
    if what == "free":
        free = len(ring) + 1
    if what == "huge counts":
        counts[:] = 2 ** 31 - 1
        lens[:] = 0
    got, d, state, st = run_tables((counts, lens, table, ring, head, free), capacity, 64, in_place=True)
    assert st == status
    assert (got.slots == -1).all() and (got.positions == -1).all() and (got.rows == -1).all() and (got.starts == 0).all()
    for x, y in zip(d, (counts, lens, table, ring)):
        assert np.array_equal(x.cpu().numpy(), y)
    assert state.tolist() == [head, free, 0, 0]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("counts, lens, free, N", [
    ([-1, 1], [64, 0], 4, 4),                    # a page returned though all are free: its place is the one that is taken
    ([-1, 64], [65, 0], 3, 4), ([-1, 64, 64], [192, 0, 0], 2, 4), ([-1] * 700 + [64] * 700, [64] * 700 + [0] * 700, 1300, 1999)])
def test_tables_refuse_more_free_pages_than_the_ring(counts, lens, free, N, in_place):
    """Returned pages that would reach round the ring into the places of the taken ones, whatever the step leaves free."""
    counts, lens = np.array(counts, np.int32), np.array(lens, np.int32)
    need = (-(-(lens + np.maximum(counts, 0)) // 64) - -(-lens // 64))[counts >= 0].sum()
    give = (-(-lens // 64))[counts < 0].sum()
    assert need <= free and free - need + give <= N < free + give
    table, ring = np.full((len(lens), 3), 1, np.int32), np.arange(N, dtype=np.int32)
    got, d, state, st = run_tables((counts, lens, table, ring, 1, free), 64 * len(lens), 64, in_place)
    assert st == bga.IKBO_ERR_PAGE_RANGE
    assert (got.slots == -1).all() and (got.rows == -1).all() and (got.starts == 0).all()
    assert np.array_equal(got.lens.cpu().numpy(), lens) and got.state.tolist()[:2] == [1, free]
    for x, y in zip(d, (counts, lens, table, ring)):
        assert np.array_equal(x.cpu().numpy(), y)


def test_tables_bad_page_numbers_give_no_slot():
    t = torch()
    step = (np.array([3, 3], np.int32), np.array([10, 64], np.int32), np.array([[77, -1], [1, -1]], np.int32), np.array([0, 99, 2, 3], np.int32), 1, 2)
    got, d, state, st = run_tables(step, 6, 64)
    assert st == bga.IKBO_ERR_PAGE_RANGE
    assert got.slots.tolist() == [-1] * 6 and got.positions.tolist() == [10, 11, 12, 64, 65, 66]
    assert got.state.dtype == t.int32


def test_tables_steps_replay_in_a_graph():
    """Twenty in-place steps as replays of one captured step, with eager work between, against the definition."""
    t = torch()
    h = H()
    rng = np.random.default_rng(3)
    B, width, N = 33, 4, 120
    table, ring = np.full((B, width), -1, np.int32), rng.permutation(N).astype(np.int32)
    lens, head, free = np.zeros(B, np.int32), 0, N
    d_table, d_ring, d_lens = dev(table), dev(ring), dev(lens)
    state, st = t.tensor([0, N, 0, 0], dtype=t.int32, device="cuda"), word()
    counts = t.zeros(B, dtype=t.int32, device="cuda")
    rows = t.empty((3, 200), dtype=t.int32, device="cuda")
    out = h.StepTables(rows[0], rows[1], rows[2], t.empty(B + 1, dtype=t.int32, device="cuda"), d_lens, state)
    side = t.cuda.Stream()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=side):
        h.kv_tables(counts, d_lens, d_table, d_ring, state, 200, st, out=out)
    t.cuda.synchronize()
    for step in range(20):
        c = rng.integers(0, 6, B).astype(np.int32)
        c[lens > 150] = -1
        counts.copy_(dev(c))
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        want = ref.tables(c, lens, table, ring, head, free, 200)
        lens, head, free = want[4], want[5], want[6]
        assert np.array_equal(rows.cpu().numpy(), np.stack(want[:3])) and np.array_equal(out.starts.cpu().numpy(), want[3]), step
        assert np.array_equal(d_lens.cpu().numpy(), lens) and state.tolist()[:2] == [head, free]
        assert np.array_equal(d_table.cpu().numpy(), table) and np.array_equal(d_ring.cpu().numpy(), ring)
    assert h.kv_status(st) == bga.IKBO_OK


def test_tables_without_rows_and_lengths_into_counts():
    t = torch()
    h = H()
    lens, counts = dev(np.array([64, 10, 0], np.int32)), t.zeros(3, dtype=t.int32, device="cuda")
    table, ring = dev(np.array([[0, -1], [1, -1], [-1, -1]], np.int32)), dev(np.array([2, 3, 4], np.int32))
    state, st = t.tensor([1, 1, 0, 0], dtype=t.int32, device="cuda"), word()
    got = h.kv_tables(counts, lens, table, ring, state, 0, st)
    assert got.slots.numel() == 0 and got.starts.tolist() == [0] * 4 and got.lens.tolist() == [64, 10, 0] and got.state.tolist()[:2] == [1, 1]
    # 40 000 rows in many blocks, the new lengths written over the counts that every block reads.
    B = 4000
    rng = np.random.default_rng(1)
    step = make_step(rng, B, 3, 64, 3, 20)
    cap = int(np.maximum(step[0], 0).sum())
    d = [dev(x) for x in step[:4]]
    state = t.tensor([step[4], step[5], 0, 0], dtype=t.int32, device="cuda")
    rows = t.empty((3, cap), dtype=t.int32, device="cuda")
    out = h.StepTables(rows[0], rows[1], rows[2], t.empty(B + 1, dtype=t.int32, device="cuda"), d[0], t.empty_like(state))
    h.kv_tables(d[0], d[1], d[2], d[3], state, cap, st, out=out)
    want = ref.tables(step[0], step[1], step[2].copy(), step[3].copy(), step[4], step[5], cap)
    assert np.array_equal(rows.cpu().numpy(), np.stack(want[:3])) and np.array_equal(d[0].cpu().numpy(), want[4])
    assert h.kv_status(st) == bga.IKBO_OK and state.tolist() == [step[4], step[5], 0, 0]


# ---- rotary positions ----------------------------------------------------------------------


def rope_case(rng, T, Hq, Hk, dim, dtype, far):
    t = torch()
    qkv = t.from_numpy(rng.standard_normal((T, Hq + 2 * Hk, dim)).astype(np.float32)).to(dtype).cuda()
    pos = rng.integers(0, far, T).astype(np.int32)
    pos[:min(T, 2)] = [0, far - 1][:min(T, 2)]
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hk], pos


@pytest.mark.parametrize("T, Hq, Hk, dim, rot", [(1, 1, 1, 2, 2), (3, 4, 2, 128, 128), (257, 3, 1, 64, 48), (5, 2, 2, 80, 20), (31, 5, 3, 10, 6),
                                                 (2, 1, 1, 1024, 1024), (9000, 2, 1, 64, 32), (7, 4, 0, 128, 64)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_rope(T, Hq, Hk, dim, rot, layout, dtype):
    t = torch()
    dt = getattr(t, dtype)
    rng = np.random.default_rng(T + dim)
    q, k, pos = rope_case(rng, T, Hq, Hk, dim, dt, 2 ** 20)
    freq, _ = H().rope_frequencies(rot, 1e4)
    p = dev(pos)
    log(f"rope T={T} heads={Hq},{Hk} dim={dim} rot={rot} {layout} {dtype}")
    for inverse, factor in ((False, 1.0), (True, 1.25)):
        qo, ko = H().rope(q, k if Hk else None, p, freq, layout=layout, factor=factor, inverse=inverse)
        for x, y in ((q, qo), (k, ko)):
            if y is None:
                continue
            want, bound = ref.turn(f64(x), pos, f64(freq), layout, factor, inverse)
            bounded(f64(y), want, bound, dt, f"{layout} inverse={inverse}")
            assert t.equal(y[..., rot:], x[..., rot:])
    only_k = H().rope(None, q, p, freq, layout=layout)
    assert only_k[0] is None and t.equal(only_k[1], H().rope(q, None, p, freq, layout=layout)[0])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_positions_over_all_of_int32(layout):
    t = torch()
    rng = np.random.default_rng(2)
    q, k, pos = rope_case(rng, 64, 2, 1, 64, t.float32, 100)
    pos[:8] = [2 ** 31 - 1, -2 ** 31, -1, 2 ** 30 + 1, 2 ** 24 + 1, -12345, 10 ** 9, 0]
    freq, _ = H().rope_frequencies(64, 1e6)
    qo, ko = H().rope(q, k, dev(pos), freq, layout=layout)
    for x, y in ((q, qo), (k, ko)):
        want, bound = ref.turn(f64(x), pos, f64(freq), layout)
        bounded(f64(y), want, bound, t.float32, layout)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_rope_in_place_and_strided(layout, dtype):
    """In place over the heads of one tensor; odd strides and bases that rule out wide accesses; neighbours untouched."""
    t = torch()
    h = H()
    dt = getattr(t, dtype)
    rng = np.random.default_rng(4)
    freq, _ = h.rope_frequencies(32, 1e4)
    pos = dev(rng.integers(0, 5000, 40).astype(np.int32))
    for pad in (0, 1, 3):
        buf = t.from_numpy(rng.standard_normal((40, 7, 64 + pad)).astype(np.float32)).to(dt).cuda()
        q, k = buf[:, 0:4, pad:], buf[:, 4:6, pad:]
        want = h.rope(q.contiguous(), k.contiguous(), pos, freq, layout=layout)
        before = buf.clone()
        out = t.full((40, 6, 70), 7.0, dtype=dt, device="cuda")
        res = h.rope(q, k, pos, freq, layout=layout, out=(out[:, :4, 1:65], out[:, 4:, 1:65]))
        assert t.equal(res[0], want[0]) and t.equal(res[1], want[1]) and (out[..., 0] == 7).all() and (out[..., 65:] == 7).all()
        assert t.equal(buf, before)
        h.rope(q, k, pos, freq, layout=layout, out=(q, k))
        assert t.equal(q, want[0]) and t.equal(k, want[1])
        assert t.equal(buf[:, 6], before[:, 6]) and t.equal(buf[..., :pad], before[..., :pad])


def test_rope_refusals():
    t = torch()
    h = H()
    x = t.zeros(6, 4, 64, dtype=t.bfloat16, device="cuda")
    p = t.zeros(6, dtype=t.int32, device="cuda")
    f = t.ones(32, dtype=t.float64, device="cuda")
    bad = [dict(q=x.half()), dict(positions=p.long()), dict(freq=f.float()), dict(layout="other"), dict(k=x.float()),
           dict(q=x.transpose(1, 2)), dict(positions=p[::2]), dict(freq=f[::2]), dict(out=(x[:, :2], x)), dict(out=(x, None))]
    for change in bad:
        with pytest.raises((ValueError, bga.IkboError)):
            h.rope(**{**dict(q=x, k=x.clone(), positions=p, freq=f), **change})
    y = t.zeros(7, 4, 64, dtype=t.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        h.rope(y[:6], None, p, f, out=(y[1:], None))
    with pytest.raises(ValueError):
        h.rope(x, None, p, f, out=(x[:1].expand(6, 4, 64), None))
    with pytest.raises(ValueError):
        h.rope(x, y[:6], p, f, out=(y[:6], x))     # each other's input
    with pytest.raises(bga.IkboError):
        h.rope(x, None, p, t.ones(33, dtype=t.float64, device="cuda"))
    e = h.rope(x[:0], None, p[:0], f)[0]
    assert e.shape == (0, 4, 64)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient(layout):
    """Against the formula's gradient, and against central differences; through expanded and shared inputs."""
    t = torch()
    from broadcast_gemm_amd.autograd import IkboRope
    rng = np.random.default_rng(6)
    T, dim, rot = 5, 20, 12
    m = IkboRope(dim, rot, 100.0, {"kind": "pairs", "factor": 4, "context": 64, "low": 1, "high": 32}, layout).cuda()
    pos = rng.integers(0, 300, T).astype(np.int32)
    q = dev(rng.standard_normal((T, 3, dim)), t.float32).requires_grad_()
    k1 = dev(rng.standard_normal((T, 1, dim)), t.float32).requires_grad_()
    wq, wk = rng.standard_normal((T, 3, dim)), rng.standard_normal((T, 2, dim))
    qo, ko = m(q, k1.expand(T, 2, dim), dev(pos))
    ((qo * dev(wq, t.float32)).sum() + (ko * dev(wk, t.float32)).sum()).backward()
    f = f64(m.freq)
    gq, bq = ref.turn(f64(dev(wq, t.float32)), pos, f, layout, m.factor, inverse=True)
    bounded(f64(q.grad), gq, bq, t.float32, "dq")
    gk, bk = ref.turn(f64(dev(wk, t.float32)), pos, f, layout, m.factor, inverse=True)
    bounded(f64(k1.grad), gk.sum(1, keepdims=True), bk.sum(1, keepdims=True) + np.abs(gk).sum(1, keepdims=True) * 2.0 ** -23, t.float32, "dk of a shared head")
    # The loss is linear in q: a difference over a step of 1 is exact but for the two sums' roundings.
    x0 = f64(q)
    for idx in ((0, 0, 0), (2, 1, rot - 1), (4, 2, rot), (3, 0, 5)):
        ends = []
        for sgn in (1, -1):
            x = x0.copy()
            x[idx] += sgn * 0.5
            ends.append((ref.turn(x, pos, f, layout, m.factor)[0] * wq).sum())
        assert abs((ends[0] - ends[1]) - float(q.grad[idx])) < 1e-5
    only_q = m(q, None, dev(pos))
    assert only_q[1] is None
    only_q[0].sum().backward()
    # The gradient is linear in the upstream gradient: differentiated again, it turns forward.
    up = dev(wq, t.float32).requires_grad_()
    g, = t.autograd.grad(m(q, None, dev(pos))[0], q, up, create_graph=True)
    gg, = t.autograd.grad(g, up, dev(wq, t.float32))
    back, bound = ref.turn(f64(dev(wq, t.float32)), pos, f, layout, m.factor)
    bounded(f64(gg), back, bound, t.float32, "gradient of the gradient")


def test_rope_module_after_casts():
    """A cast of the module, before or after it moves to the GPU, changes no rotation."""
    t = torch()
    from broadcast_gemm_amd.autograd import IkboRope
    rng = np.random.default_rng(27)
    q = dev(rng.standard_normal((9, 3, 64)), t.bfloat16)
    pos = dev(rng.integers(0, 10 ** 6, 9).astype(np.int32))
    want = IkboRope(64, 32).cuda()(q, None, pos)[0]
    for m in (IkboRope(64, 32).bfloat16().cuda(), IkboRope(64, 32).cuda().half(), IkboRope(64, 32).to("cuda", t.bfloat16).float()):
        assert t.equal(m(q, None, pos)[0], want)


def test_rope_gradient_replays_in_a_graph():
    """Forward and backward captured together, with leaves that no eager graph holds; every replay against an eager pass."""
    t = torch()
    from broadcast_gemm_amd.autograd import IkboRope
    rng = np.random.default_rng(26)
    m = IkboRope(64, 32).cuda()
    pos = t.zeros(33, dtype=t.int32, device="cuda")
    q, up = (t.zeros(33, 3, 64, device="cuda") for _ in range(2))
    q.requires_grad_()
    graph = t.cuda.CUDAGraph()
    t.cuda.synchronize()
    with t.cuda.graph(graph):
        turned = m(q, None, pos)[0]
        grad, = t.autograd.grad(turned, q, up)
    for rep in range(4):
        eager = dev(rng.standard_normal((33, 3, 64)), t.float32).requires_grad_()
        with t.no_grad():
            q.copy_(eager)
        up.copy_(dev(rng.standard_normal((33, 3, 64)), t.float32))
        pos.copy_(dev(rng.integers(0, 5000, 33).astype(np.int32)))
        want = m(eager, None, pos)[0]
        want_grad, = t.autograd.grad(want, eager, up)
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(turned, want) and t.equal(grad, want_grad), rep


def test_rope_more_tokens_than_one_launch_counts():
    """2^24 tokens and a few, heads that leave one token to a block: over 2^32 threads."""
    t = torch()
    T = (1 << 24) + 5
    log(f"rope T={T}")
    x = t.linspace(-2, 2, 258, device="cuda").to(t.bfloat16).view(1, 1, 258)
    pos = t.zeros(T, dtype=t.int32, device="cuda")
    pos[0], pos[-3], pos[-1] = 1, 2, 3
    freq = H().rope_frequencies(258)[0]
    out = t.zeros(T, 1, 258, dtype=t.bfloat16, device="cuda")
    H().rope(x.expand(T, 1, 258), None, pos, freq, out=(out, None))
    turned = H().rope(x.expand(4, 1, 258), None, t.arange(4, dtype=t.int32, device="cuda"), freq)[0]
    assert t.equal(turned[0], x[0])
    assert t.equal(out[0], turned[1]) and t.equal(out[-3], turned[2]) and t.equal(out[-1], turned[3])
    out[0] = out[-3] = out[-1] = x[0]
    assert all(bool((part == x).all()) for part in out.split(1 << 21))


# ---- the cache: write and read -------------------------------------------------------------


def cache(pages, heads, dim, fill=0):
    t = torch()
    return t.full((pages, heads, 68 * dim), fill, dtype=t.uint8, device="cuda")


def check_write(k, v, slots, pages, heads, dim, fill=0x5A):
    """Bytes of every tile against the definition, untouched ones included; then the values read back."""
    t = torch()
    tiles, st = cache(pages, heads, dim, fill), word()
    want = tiles.cpu().numpy()
    H().kv4_write(k, v, dev(slots), tiles, st)
    ref.put(want, f64(k), f64(v), slots)
    assert H().kv_status(st) == bga.IKBO_OK
    got = tiles.cpu().numpy()
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"
    kv = ref.rows_of(want)
    live = slots >= 0
    for dt in (t.bfloat16, t.float32):
        out = tuple(t.full((len(slots), heads, dim), 9.0, dtype=dt, device="cuda") for _ in range(2))
        H().kv4_read(dev(slots), tiles, st, out=out)
        for x, y in zip(out, kv):
            x = f64(x)
            assert np.array_equal(x[live], y[slots[live] // 64, :, slots[live] % 64])
            assert (x[~live] == 9).all()
    assert H().kv_status(st) == bga.IKBO_OK


@pytest.mark.parametrize("T, heads, dim, order", [(1, 1, 64, "run"), (1, 3, 128, "random"), (59, 4, 128, "random"), (64, 2, 64, "run"), (65, 1, 128, "run"),
                                                  (200, 2, 64, "offset"), (333, 2, 128, "offset"), (130, 1, 64, "reverse"), (150, 3, 128, "random")])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_write_and_read(T, heads, dim, order, dtype):
    t = torch()
    rng = np.random.default_rng(T + dim)
    pages = T // 64 + 3
    x = rng.standard_normal((2, T, heads, dim)) * np.exp(2 * rng.standard_normal((2, T, heads, 1)))
    kv = dev(x, getattr(t, dtype))
    slots = {"run": np.arange(T), "offset": np.arange(T) + 37, "reverse": np.arange(T)[::-1] + 5,
             "random": rng.permutation(pages * 64)[:T]}[order].astype(np.int32)
    if T > 20:
        slots[[3, 17, T - 1]] = -1
    log(f"write T={T} heads={heads} dim={dim} {order} {dtype}")
    check_write(kv[0], kv[1], slots, pages, heads, dim)


@pytest.mark.parametrize("T, heads, dim, order", [
    (4032, 8, 128, "offset"),      # 504 blocks of 64 rows: the last step that takes 16 rows a block
    (4033, 8, 128, "offset"), (4033, 8, 64, "run"), (4160, 8, 128, "run"), (4103, 8, 64, "offset"), (4103, 8, 128, "random"), (4103, 8, 64, "random"),
    (4219, 8, 128, "runs"), (4219, 8, 64, "runs"), (4103, 8, 128, "reverse"), (4103, 8, 64, "reverse"), (1, 512, 64, "run"), (70, 257, 128, "offset")])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_write_and_read_blocks_of_64_rows(T, heads, dim, order, dtype):
    """Steps of many rows, on both sides of the rule that takes 64 rows to a block: whole runs, runs that start and end
    inside a page and inside a block, and rows without neighbours; every byte, then the values read back."""
    t = torch()
    rng = np.random.default_rng(T + dim)
    pages = T // 64 + 3
    x = dev(rng.standard_normal((2, T, heads, dim)) * np.exp(2 * rng.standard_normal((2, T, heads, 1))), getattr(t, dtype))
    slots = {"run": np.arange(T), "offset": np.arange(T) + 37, "reverse": np.arange(T)[::-1] + 5, "random": rng.permutation(pages * 64)[:T],
             "runs": None}[order]
    if order == "runs":            # pieces of 1 to 40 slots in random order
        cuts = np.cumsum(rng.integers(1, 41, pages * 64))
        pieces = np.split(np.arange(pages * 64), cuts[cuts < pages * 64])
        slots = np.concatenate([pieces[i] for i in rng.permutation(len(pieces))])[:T]
    slots = slots.astype(np.int32)
    if T > 20:
        slots[[3, 17, T // 2, T - 1]] = -1
    log(f"write in blocks of 64: T={T} heads={heads} dim={dim} {order} {dtype}")
    tiles, st = cache(pages, heads, dim, 0x5A), word()
    want = tiles.cpu().numpy()
    d_slots = dev(slots)
    H().kv4_write(x[0], x[1], d_slots, tiles, st)
    ref.put_all(want, f64(x[0]), f64(x[1]), slots)
    assert H().kv_status(st) == bga.IKBO_OK
    got = tiles.cpu().numpy()
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"
    live = slots >= 0
    values = ref.rows_of(want)
    for dt in (t.bfloat16, t.float32):
        out = tuple(t.full((T, heads, dim), 9.0, dtype=dt, device="cuda") for _ in range(2))
        H().kv4_read(d_slots, tiles, st, out=out)
        for o, y in zip(out, values):
            o = f64(o)
            assert np.array_equal(o[live], y[slots[live] // 64, :, slots[live] % 64]) and (o[~live] == 9).all()
    assert H().kv_status(st) == bga.IKBO_OK


def test_write_strided_rows():
    t = torch()
    rng = np.random.default_rng(8)
    qkv = dev(rng.standard_normal((70, 6, 72)), t.bfloat16)
    k, v = qkv[:, 2:4, :64], qkv[:, 4:6, 8:]
    check_write(k, v, (rng.permutation(256)[:70]).astype(np.int32), 4, 2, 64)
    check_write(k[:1].expand(70, 2, 64), v, (rng.permutation(256)[:70]).astype(np.int32), 4, 2, 64)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_write_every_code_border_and_magnitude(dtype):
    """Values on, just below and just above every rounding border, at scales from the smallest to the largest."""
    t = torch()
    dt = getattr(t, dtype)
    borders = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6])
    step = 2.0 ** -7 if dtype == "bfloat16" else 2.0 ** -22
    vals = np.concatenate([borders, borders * (1 + step), borders * (1 - step)])
    vals = vals[vals <= 6]
    exps = [-133, -126, -125, -124, -60, -1, 0, 1, 60, 123, 124, 125]
    rows = []
    for e in exps:
        for top in (6.0, 5.0, 3.0 * (1 + 2 * step), 3.0, 4.0):
            for i in range(0, len(vals), 31):
                b = np.zeros(32)
                part = np.minimum(vals[i:i + 31], top)
                b[:len(part)] = part * np.where(np.arange(len(part)) % 2, -1, 1)
                b[31] = top
                rows.append(b * 2.0 ** e)
    rows = np.array(rows + [np.zeros(32)] * (-len(rows) % 4))
    x = t.from_numpy(rows.reshape(-1, 1, 128).astype(np.float32)).to(dt).cuda()
    T = x.shape[0]
    check_write(x, x.flip(0).contiguous(), np.arange(T, dtype=np.int32), T // 64 + 1, 1, 128)


def test_write_marks_what_the_format_cannot_hold():
    t = torch()
    h = H()
    for bad, value in ((float("inf"), 6 * 2.0 ** 125), (float("-inf"), -6 * 2.0 ** 125), (float("nan"), 0.0)):
        k = t.zeros(3, 1, 64, dtype=t.float32, device="cuda")
        k[1, 0, 40] = bad
        v = t.ones_like(k)
        tiles, st = cache(1, 1, 64), word()
        slots = dev(np.array([0, 1, 2], np.int32))
        h.kv4_write(k, v, slots, tiles, st)
        assert h.kv_status(st) == bga.IKBO_ERR_NONFINITE and h.kv_status(st) == bga.IKBO_OK
        kk, vv = h.kv4_read(slots, tiles, st, dtype=t.float32)
        want = t.zeros_like(k)
        want[1, 0, 40] = value
        assert t.equal(kk, want) and t.equal(vv, v)


def test_write_and_read_bad_slots():
    t = torch()
    h = H()
    k = t.ones(4, 2, 64, dtype=t.bfloat16, device="cuda")
    for slot in (128, -2, 2 ** 31 - 1, -2 ** 31):
        tiles, st = cache(2, 2, 64, 3), word()
        slots = dev(np.array([0, slot, 127, -1], np.int32))
        h.kv4_write(k, k, slots, tiles, st)
        assert h.kv_status(st) == bga.IKBO_ERR_PAGE_RANGE
        out = tuple(t.full_like(k, 5.0) for _ in range(2))
        h.kv4_read(slots, tiles, st, out=out)
        assert h.kv_status(st) == bga.IKBO_ERR_PAGE_RANGE
        for o in out:
            assert (o[[0, 2]] == 1).all() and (o[[1, 3]] == 5).all()


def test_rows_refusals():
    t = torch()
    h = H()
    k = t.ones(4, 2, 64, dtype=t.bfloat16, device="cuda")
    slots, tiles, st = dev(np.arange(4, dtype=np.int32)), cache(2, 2, 64), word()
    for args in ((k.half(), k.half()), (k, k.float()), (k[:3], k), (k[:, :1], k), (k.transpose(1, 2), k), (k[..., ::2], k)):
        with pytest.raises((ValueError, bga.IkboError)):
            h.kv4_write(*args, slots, tiles, st)
    odd = t.ones(4, 2, 68, dtype=t.bfloat16, device="cuda")
    with pytest.raises(bga.IkboError):
        h.kv4_write(odd[..., :64], k, slots, tiles, st)
    with pytest.raises(ValueError):
        h.kv4_write(k, k, slots.long(), tiles, st)
    with pytest.raises(ValueError):
        h.kv4_read(slots, tiles, st, dtype=t.float16)
    with pytest.raises((ValueError, bga.IkboError)):
        h.kv4_read(slots, tiles[..., :-1], st)
    h.kv4_write(k[:0], k[:0], slots[:0], tiles, st)
    assert h.kv4_read(slots[:0], tiles, st)[0].shape == (0, 2, 64) and not tiles.any()


@pytest.mark.parametrize("T, op", [((1 << 30) + 70, "write"), ((1 << 29) + 70, "read")])
def test_more_rows_than_one_launch_counts(T, op):
    """Rows whose launch would have over 2^32 threads, all padding but a few at both ends, each the same row in memory
    (strides of 0; a read's rows hold equal values)."""
    import ctypes
    from test_history import _RowsArgs, fill
    t = torch()
    log(f"{op} T={T}")
    slots = t.full((T,), -1, dtype=t.int32, device="cuda")
    first = t.tensor([5, 6, 7, 8, 9], dtype=t.int32, device="cuda")
    slots[:5], slots[-3:] = first, t.tensor([70, 71, 3], dtype=t.int32, device="cuda")
    kv = t.linspace(-6, 6, 128, device="cuda").view(2, 1, 1, 64)
    tiles, st = cache(2, 1, 64), word()
    few = t.cat([first, slots[-3:]])
    H().kv4_write(*(x.expand(8, 1, 64) for x in kv), few, tiles, st)
    want_k, want_v = H().kv4_read(few, tiles, st, dtype=t.float32)
    got_tiles = tiles if op == "read" else t.zeros_like(tiles)
    rows = t.zeros_like(kv) if op == "read" else kv
    if op == "read":                      # the last row alone decides what is left
        slots[:5] = -1
    args = fill(_RowsArgs, k=rows[0].data_ptr(), v=rows[1].data_ptr(), slots=slots.data_ptr(), tiles=got_tiles.data_ptr(), status=st.data_ptr(),
                k_token=0, k_head=64, v_token=0, v_head=64, T=T, H_kv=1, head_dim=64, num_pages=2, dtype=1)
    t.cuda.synchronize()
    assert getattr(bga.lib(), "ikbo_kv4_" + op)(ctypes.byref(args), None) == bga.IKBO_OK
    assert H().kv_status(st) == bga.IKBO_OK
    assert t.equal(got_tiles, tiles)
    assert t.equal(rows[0, 0], want_k[0] if op == "read" else kv[0, 0]) and t.equal(rows[1, 0], want_v[0] if op == "read" else kv[1, 0])


def test_slots_past_32_bits_of_bytes():
    t = torch()
    pages = (1 << 32) // (68 * 64) + 50
    tiles, st = t.empty((pages, 1, 68 * 64), dtype=t.uint8, device="cuda"), word()
    rng = np.random.default_rng(9)
    kv = dev(rng.standard_normal((2, 6, 1, 64)), t.bfloat16)
    slots = np.array([5, (pages - 1) * 64 + 63, (pages - 1) * 64, (pages - 40) * 64 + 7, (pages - 41) * 64, 64], np.int32)
    H().kv4_write(kv[0], kv[1], dev(slots), tiles, st)
    got = H().kv4_read(dev(slots), tiles, st, dtype=t.float32)
    for x, y in zip(got, kv):
        assert np.array_equal(f64(x), ref.decode(*ref.encode(f64(y))))
    # The same rows as a history, attended over: page numbers of the far end.
    lens, table = dev(np.array([1], np.int32)), dev(np.array([[pages - 40]], np.int32))
    H().kv4_write(kv[0][3:4], kv[1][3:4], dev(np.array([(pages - 40) * 64], np.int32)), tiles, st)
    O = H().kv4_attention(kv[0][:1].contiguous(), tiles, table, lens, None, st)
    assert np.array_equal(f64(O)[0, 0], f64(got[1])[3, 0]) and H().kv_status(st) == bga.IKBO_OK


# ---- attention -----------------------------------------------------------------------------


def history(rng, lens, width, heads, dim, junk=True):
    """Tiles (random codes, scales 2^-3 .. 2^0; past the histories and in unused pages bytes of 255), table, and the values."""
    t = torch()
    need = -(-lens // 64)
    pages = int(need.sum()) + 2
    order = rng.permutation(pages)
    table = np.full((len(lens), width), -1, np.int32)
    tiles = rng.integers(0, 256, (pages, heads, 68 * dim)).astype(np.uint8)
    tiles[..., 64 * dim:] = rng.integers(124, 128, (pages, heads, 4 * dim))
    at = 0
    for u, n in enumerate(need):
        table[u, :n] = order[at:at + n]
        at += n
    k, v = ref.rows_of(tiles)
    if junk:
        tiles[order[at:]] = 255
        for u, n in enumerate(lens):
            if n % 64:
                w = tiles[table[u, n // 64]]
                past = np.arange(n % 64, 64)
                w[:, 64 * dim:66 * dim].reshape(heads, dim // 32, 64)[..., ref.scale_place(past)] = 255
                w[:, 66 * dim:].reshape(heads, dim // 32, 64)[..., past] = 255
    return t.from_numpy(tiles).cuda(), dev(table), table, k, v


def attend_case(seed, lens, B_c, Hq, Hkv, Lq, dim, mapping="even", positions=False, width=None, scale=0.0):
    rng = np.random.default_rng(seed)
    t = torch()
    lens = np.asarray(lens)
    B_u = len(lens)
    width = width or max(1, int(-(-lens.max() // 64)))
    tiles, d_table, table, k, v = history(rng, lens, width, Hkv, dim)
    mp = {"even": np.arange(B_c) * B_u // max(1, B_c), "random": rng.integers(0, B_u, B_c), "none": None}[mapping]
    pos = None
    if positions:
        pos = rng.integers(-1, max(2, lens.max() + 3), (B_c, Lq)).astype(np.int32)
    Q = dev(rng.standard_normal((B_c, Hq, Lq, dim)) * 1.5, t.bfloat16)
    st = word()
    d_mp = None if mp is None else dev(mp.astype(np.int32))
    d_pos = None if pos is None else dev(pos)
    O = H().kv4_attention(Q, tiles, d_table, dev(lens.astype(np.int32)), d_mp, st, positions=d_pos, scale=scale)
    want, bound = ref.attend(f64(Q), k, v, table, lens, mp, pos, scale or None)
    bounded(f64(O), want, bound, t.bfloat16, f"lens={lens.tolist()[:8]} B_c={B_c} heads={Hq}/{Hkv} L_q={Lq} dim={dim}")
    assert H().kv_status(st) == bga.IKBO_OK
    again = H().kv4_attention(Q, tiles, d_table, dev(lens.astype(np.int32)), d_mp, st, positions=d_pos, scale=scale)
    assert t.equal(O, again)
    return O


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens, Hq, Hkv", [([1], 1, 1), ([0], 2, 1), ([64], 1, 1), ([65], 3, 1), ([63, 0, 1], 4, 2), ([200, 7, 128, 129], 8, 2),
                                           ([1000, 3], 16, 1), ([130, 2000, 0, 64], 32, 8), ([4000], 20, 1), ([77] * 40, 6, 3)])
def test_attend_one_token(lens, Hq, Hkv, dim):
    """One query token per user: short and long histories, empty ones, shared key heads from none to 20."""
    log(f"attend one token lens={lens[:4]} heads={Hq}/{Hkv} dim={dim}")
    attend_case(len(lens) + dim, lens, len(lens), Hq, Hkv, 1, dim, mapping="none")


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens, B_c, Hq, Hkv, Lq, mapping", [
    ([100, 50], 7, 2, 2, 3, "even"), ([64, 129, 0], 30, 2, 1, 5, "random"), ([300], 9, 4, 2, 16, "even"), ([90, 10, 700], 12, 1, 1, 33, "random"),
    ([500, 20], 5, 2, 1, 64, "even"), ([31, 64, 65, 1], 100, 3, 3, 1, "random"), ([64] * 70, 71, 1, 1, 2, "random"), ([250, 40], 3, 5, 1, 7, "even")])
def test_attend_targets(lens, B_c, Hq, Hkv, Lq, mapping, dim):
    """Candidates over their users' histories: sorted and unsorted maps, users without candidates, odd query counts."""
    log(f"attend targets lens={lens[:4]} B_c={B_c} heads={Hq}/{Hkv} L_q={Lq} {mapping} dim={dim}")
    attend_case(B_c + dim, lens, B_c, Hq, Hkv, Lq, dim, mapping=mapping)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens, B_c, Hq, Hkv, Lq, mapping", [([150, 64, 3], 40, 4, 2, 1, "even"), ([300, 0, 65], 9, 2, 1, 6, "random"),
                                                             ([1], 3, 2, 2, 4, "even"), ([700, 700], 60, 3, 1, 1, "random")])
def test_attend_positions(lens, B_c, Hq, Hkv, Lq, mapping, dim):
    """Queries limited by position: from none (-1) to past the history's end."""
    log(f"attend positions lens={lens[:4]} B_c={B_c} heads={Hq}/{Hkv} L_q={Lq} dim={dim}")
    attend_case(B_c * dim, lens, B_c, Hq, Hkv, Lq, dim, mapping=mapping, positions=True)


@pytest.mark.parametrize("B_u, B_c, Hq, Hkv, Lq, dim, longest, mapping, positions", [
    (300, 300, 4, 2, 1, 64, 200, "none", False),        # more users than a block's own plan holds
    (2500, 2400, 2, 1, 1, 64, 130, "none", False),
    (4096, 4096, 1, 1, 1, 64, 70, "random", True),
    (257, 3000, 1, 1, 1, 128, 300, "random", False),
    (2, 1025, 1, 1, 1, 64, 500, "random", True),         # many rows: the wide kernel, rows limited by position
    (3, 1200, 2, 1, 1, 64, 900, "even", True),
    (5, 900, 3, 3, 2, 128, 333, "random", False),
    (1, 700, 1, 1, 1, 128, 4500, "even", True),          # long enough to be cut in many runs
    (1, 64, 4, 1, 2, 128, 9000, "even", False),
    (2, 2, 16, 1, 1, 64, 20000, "none", False),          # more than 64 pieces to join
    (1, 1, 1, 1, 1, 128, 30000, "none", False),
    (7, 50, 2, 1, 1, 128, 40, "random", False)])
def test_attend_plans(B_u, B_c, Hq, Hkv, Lq, dim, longest, mapping, positions):
    """Every way the work is planned, dealt and joined; a sample of the candidates against the definition."""
    t = torch()
    log(f"attend plan B_u={B_u} B_c={B_c} heads={Hq}/{Hkv} L_q={Lq} dim={dim} longest={longest} {mapping} {positions}")
    rng = np.random.default_rng(B_u + B_c)
    lens = rng.integers(0, longest + 1, B_u)
    lens[rng.integers(0, B_u)] = longest
    if B_u > 5:
        lens[rng.random(B_u) < 0.1] = 0
    width = -(-longest // 64)
    tiles, d_table, table, k, v = history(rng, lens, width, Hkv, dim)
    mp = {"even": np.arange(B_c) * B_u // B_c, "random": rng.integers(-1, B_u, B_c), "none": None}[mapping]
    pos = rng.integers(-1, longest + 3, (B_c, Lq)).astype(np.int32) if positions else None
    Q = dev(rng.standard_normal((B_c, Hq, Lq, dim)) * 1.5, t.bfloat16)
    st = word()
    out = t.full_like(Q, 5.0)
    H().kv4_attention(Q, tiles, d_table, dev(lens.astype(np.int32)), None if mp is None else dev(mp.astype(np.int32)), st,
                      positions=None if pos is None else dev(pos), out=out)
    assert H().kv_status(st) == bga.IKBO_OK
    pick = np.unique(np.concatenate([[0, B_c - 1], rng.integers(0, B_c, 40)]))
    users = np.arange(B_c) if mp is None else mp
    want, bound = ref.attend(f64(Q)[pick], k, v, table, lens, users[pick], None if pos is None else pos[pick])
    got = f64(out)
    live = users[pick] >= 0
    bounded(got[pick][live], want[live], bound[live], t.bfloat16, "sampled candidates")
    assert (got[users < 0] == 5).all() and np.isfinite(got).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("B_u, Hkv, width", [(5, 2, 16500), (300, 1, 220)])
def test_attend_tables_for_more_than_the_last_cache_level(B_u, Hkv, width, dim):
    """Tables whose histories could take more than 256 MB: tiles are read past the caches then."""
    assert B_u * width * Hkv * 68 * dim > 256 << 20
    lens = list(np.random.default_rng(width).integers(0, 200, B_u))
    attend_case(5, lens, B_u, 2 * Hkv, Hkv, 2, dim, mapping="none", width=width)


@pytest.mark.parametrize("dim", [64, 128])
def test_attend_units_that_see_nothing(dim):
    """Many rows of one page each, several units to a block; whole units and parts of them see no token."""
    t = torch()
    rng = np.random.default_rng(dim)
    B_c, Hkv, lens = 40000, 4, np.array([50])
    tiles, d_table, table, k, v = history(rng, lens, 1, Hkv, dim)
    pos = np.where(np.arange(B_c) // 256 % 3 < 2, -1, rng.integers(-1, 60, B_c)).astype(np.int32)[:, None]
    pos[300:310] = 20
    Q = dev(rng.standard_normal((B_c, Hkv, 1, dim)), t.bfloat16)
    st = word()
    out = t.full_like(Q, 5.0)
    H().kv4_attention(Q, tiles, d_table, dev(lens.astype(np.int32)), dev(np.zeros(B_c, np.int32)), st, positions=dev(pos), out=out)
    assert H().kv_status(st) == bga.IKBO_OK
    got = f64(out)
    pick = np.unique(np.concatenate([np.arange(290, 320), rng.integers(0, B_c, 60)]))
    want, bound = ref.attend(f64(Q)[pick], k, v, table, lens, np.zeros(len(pick), int), pos[pick])
    bounded(got[pick], want, bound, t.bfloat16, "sampled candidates")
    assert (got[pos[:, 0] < 0] == 0).all()


def test_attend_scale_and_wide_table():
    attend_case(1, [100, 700], 2, 4, 2, 1, 128, mapping="none", scale=0.31, width=50)
    attend_case(2, [100, 700], 2, 4, 2, 1, 64, mapping="none", scale=3.0)


@pytest.mark.parametrize("scale", [1e-38, 1e-42, 1e-50, 5e-324])
def test_attend_scales_below_float32(scale):
    """A positive scale too small for float32 is no scale of 0, which means the default: all weights are equal."""
    attend_case(91, [150, 64], 6, 2, 1, 1, 64, mapping="random", scale=scale)


def test_attend_layouts_padding_and_untouched_rows():
    """Q and O as views of token-major buffers; padding candidates and everything around O keep their bytes."""
    t = torch()
    rng = np.random.default_rng(11)
    lens = np.array([70, 0, 130])
    tiles, d_table, table, k, v = history(rng, lens, 3, 2, 64)
    B_c, Hq, Lq = 9, 4, 5
    mp = np.array([2, -1, 0, 1, 2, -1, 0, 0, -1])
    qbuf = dev(rng.standard_normal((B_c, Lq, 3 * Hq, 64)), t.bfloat16)
    Q = qbuf[:, :, Hq:2 * Hq].transpose(1, 2)
    obuf = t.full((B_c, Lq, Hq + 2, 72), 5.0, dtype=t.bfloat16, device="cuda")
    O = obuf[:, :, 1:Hq + 1, :64].transpose(1, 2)
    st = word()
    H().kv4_attention(Q, tiles, d_table, dev(lens.astype(np.int32)), dev(mp.astype(np.int32)), st, out=O)
    want, bound = ref.attend(f64(Q), k, v, table, lens, mp, None)
    live = mp >= 0
    bounded(f64(O)[live], want[live], bound[live], t.bfloat16, "strided")
    assert (O[~dev(live)] == 5).all()
    rest = obuf.clone()
    rest[:, :, 1:Hq + 1, :64] = 5.0
    assert (rest == 5).all() and H().kv_status(st) == bga.IKBO_OK
    q3 = Q[:, :, 0]
    o3 = H().kv4_attention(q3, tiles, d_table, dev(lens.astype(np.int32)), dev(mp.astype(np.int32)), st)
    assert t.equal(o3[dev(live)], O[:, :, 0][dev(live)])


def test_attend_reports_bad_maps_lengths_and_pages():
    t = torch()
    rng = np.random.default_rng(12)
    lens = np.array([100, 64])
    tiles, d_table, table, k, v = history(rng, lens, 2, 1, 64)
    Q = dev(rng.standard_normal((4, 1, 1, 64)), t.bfloat16)
    d_lens, st = dev(lens.astype(np.int32)), word()
    out = t.full_like(Q, 5.0)
    H().kv4_attention(Q, tiles, d_table, d_lens, dev(np.array([0, 2, 1, -7], np.int32)), st, out=out)
    assert H().kv_status(st) == bga.IKBO_ERR_MAP_RANGE
    want, bound = ref.attend(f64(Q), k, v, table, lens, np.array([0, -1, 1, -1]), None)
    bounded(f64(out)[[0, 2]], want[[0, 2]], bound[[0, 2]], t.bfloat16, "valid candidates")
    assert (out[[1, 3]] == 5).all()
    mp = dev(np.array([0, 0, 1, 1], np.int32))
    for bad in (-5, 129, 2 ** 31 - 1):
        H().kv4_attention(Q, tiles, d_table, dev(np.array([100, bad], np.int32)), mp, st, out=out)
        assert H().kv_status(st) == bga.IKBO_ERR_PAGE_RANGE
        bounded(f64(out)[:2], ref.attend(f64(Q), k, v, table, lens, np.array([0, 0, -1, -1]), None)[0][:2], bound[:1], t.bfloat16, "the other user")
    for bad in (-1, len(k), 2 ** 31 - 1):
        wrong = d_table.clone()
        wrong[1, 0] = bad
        H().kv4_attention(Q, tiles, wrong, d_lens, mp, st, out=out)
        assert H().kv_status(st) == bga.IKBO_ERR_PAGE_RANGE


def test_attend_infinite_and_nan_queries_stay_in_their_rows():
    t = torch()
    rng = np.random.default_rng(13)
    lens = np.array([150])
    tiles, d_table, table, k, v = history(rng, lens, 3, 1, 128)
    Q = dev(rng.standard_normal((1, 1, 20, 128)), t.bfloat16)
    st = word()
    args = (tiles, d_table, dev(lens.astype(np.int32)), None, st)
    good = H().kv4_attention(Q, *args)
    bad = Q.clone()
    bad[0, 0, 3, 5] = float("nan")
    bad[0, 0, 17] = float("inf")
    got = H().kv4_attention(bad, *args)
    keep = [i for i in range(20) if i not in (3, 17)]
    assert t.equal(got[0, 0, keep], good[0, 0, keep]) and got[0, 0, 3].isnan().all()


def test_attend_large_scores_and_constant_rows():
    """Scores of thousands, far apart, and all equal: the maximum moves, weights neither overflow nor vanish."""
    t = torch()
    rng = np.random.default_rng(14)
    lens = np.array([500])
    tiles, d_table, table, k, v = history(rng, lens, 8, 1, 64)
    for factor in (0.0, 300.0):
        Q = dev(rng.standard_normal((1, 1, 9, 64)) * factor, t.bfloat16)
        st = word()
        O = H().kv4_attention(Q, tiles, d_table, dev(lens.astype(np.int32)), None, st)
        want, bound = ref.attend(f64(Q), k, v, table, lens, None, None)
        bounded(f64(O), want, bound, t.bfloat16, f"factor {factor}")


def test_attend_strides_past_32_bits():
    t = torch()
    rng = np.random.default_rng(15)
    lens = np.array([70, 64])
    tiles, d_table, table, k, v = history(rng, lens, 2, 1, 64)
    far = (1 << 31) + 64
    q = dev(rng.standard_normal((2, 1, 1, 64)), t.bfloat16)
    big = t.empty(far + 64, dtype=t.bfloat16, device="cuda")
    Q = big.as_strided((2, 1, 1, 64), (far, 64, 64, 1))
    Q.copy_(q)
    st = word()
    want = H().kv4_attention(q, tiles, d_table, dev(lens.astype(np.int32)), None, st)
    got = H().kv4_attention(Q, tiles, d_table, dev(lens.astype(np.int32)), None, st, out=Q)
    assert t.equal(got, want)


@pytest.mark.parametrize("B_u, B_c, Lq, n, dim", [(2, 12, 64, 1500, 64), (1, 1, 1, 9000, 128), (3, 40, 5, 300, 128)])
def test_attend_over_its_queries_and_replayed(B_u, B_c, Lq, n, dim):
    """O written over Q (also where units are cut), and the call captured and replayed with other queries between."""
    t = torch()
    rng = np.random.default_rng(16)
    lens = np.full(B_u, n)
    tiles, d_table, table, k, v = history(rng, lens, -(-n // 64), 2, dim)
    mp = dev((np.arange(B_c) % B_u).astype(np.int32))
    st, d_lens = word(), dev(lens.astype(np.int32))
    Q = t.zeros(B_c, 4, Lq, dim, dtype=t.bfloat16, device="cuda")
    graph = t.cuda.CUDAGraph()
    t.cuda.synchronize()
    with t.cuda.graph(graph):
        O = H().kv4_attention(Q, tiles, d_table, d_lens, mp, st)
    for rep in range(4):
        q = dev(rng.standard_normal(tuple(Q.shape)), t.bfloat16)
        want = H().kv4_attention(q, tiles, d_table, d_lens, mp, st)
        Q.copy_(q)
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(O, want), rep
        same = q.clone()
        assert H().kv4_attention(same, tiles, d_table, d_lens, mp, st, out=same) is not None and t.equal(same, want)
    assert H().kv_status(st) == bga.IKBO_OK


def test_attend_refusals():
    t = torch()
    h = H()
    Q = t.zeros(3, 4, 2, 64, dtype=t.bfloat16, device="cuda")
    tiles, st = cache(4, 2, 64), word()
    table, lens = t.zeros(3, 2, dtype=t.int32, device="cuda"), t.zeros(3, dtype=t.int32, device="cuda")
    ok = dict(Q=Q, tiles=tiles, block_table=table, lens=lens, mp=lens, status=st)
    for change in (dict(Q=Q.float()), dict(Q=Q[:, :3]), dict(Q=Q[..., :32]), dict(lens=lens.long()), dict(mp=lens[:2]), dict(mp=lens.long()),
                   dict(positions=lens), dict(block_table=table[:2]), dict(block_table=table.long()), dict(scale=-1.0), dict(scale=float("nan")),
                   dict(status=lens), dict(tiles=tiles.int()), dict(out=Q.float()), dict(out=Q[:1].expand(3, 4, 2, 64)), dict(Q=Q.transpose(2, 3))):
        with pytest.raises((ValueError, bga.IkboError)):
            h.kv4_attention(**{**ok, **change})
    four = t.zeros(4, 4, 2, 64, dtype=t.bfloat16, device="cuda")
    with pytest.raises(bga.IkboError):
        h.kv4_attention(four, tiles, table, lens, None, st)
    assert h.kv4_attention(Q[:0], tiles, table, lens, lens[:0], st).shape == (0, 4, 2, 64)
    assert (h.kv4_attention(**ok) == 0).all()     # lengths 0


# ---- together ------------------------------------------------------------------------------


def test_histories_grow_and_are_attended():
    """Steps of arrivals, growth and leaving through UserHistories, rotary keys and queries; each step's attention
    (candidates, and the users' own new tokens causally) against the definition over the cached values."""
    t = torch()
    h = H()
    rng = np.random.default_rng(20)
    users, Hkv, Hq, dim = 6, 2, 4, 64
    hist = h.UserHistories(users, 320, 24, Hkv, dim, rot_dim=48, theta=1000.0)
    lens = np.zeros(users, int)
    f = f64(hist.freq)
    held = [([], []) for _ in range(users)]   # the cached values by the definition
    for step, counts in enumerate(([70, 3, 0, 64, 1, 130], [1, 1, 1, 1, 1, 1], [5, -1, 80, -1, 0, 1], [1, 64, 1, 100, 1, 1])):
        counts = np.array(counts)
        new = np.maximum(counts, 0)
        T = int(new.sum()) + 3
        k, v = (dev(rng.standard_normal((T, Hkv, dim)), t.bfloat16) for _ in range(2))
        tab = hist.append(k, v, dev(counts.astype(np.int32)))
        at = 0
        for u in range(users):
            if counts[u] < 0:
                held[u], lens[u] = ([], []), 0
                continue
            pos = np.arange(lens[u], lens[u] + new[u], dtype=np.int32)
            turned = h.rope(None, k[at:at + new[u]], dev(pos), hist.freq)[1]
            want, bound = ref.turn(f64(k[at:at + new[u]]), pos, f, "half")
            bounded(f64(turned), want, bound, t.bfloat16, "turned keys")
            held[u][0].extend(ref.decode(*ref.encode(f64(turned))))
            held[u][1].extend(ref.decode(*ref.encode(f64(v[at:at + new[u]]))))
            at += new[u]
            lens[u] += new[u]
        assert np.array_equal(hist.lens.cpu().numpy(), lens) and hist.check() == bga.IKBO_OK
        # The cached values as one page set per user, for the plain form.
        kp, vp = (np.zeros((users * 5, Hkv, 64, dim)) for _ in range(2))
        table = np.arange(users * 5).reshape(users, 5)
        for u in range(users):
            for dst, src in ((kp, held[u][0]), (vp, held[u][1])):
                for i, row in enumerate(src):
                    dst[u * 5 + i // 64, :, i % 64] = row
        # Candidates of random users, standing behind the histories.
        mp = rng.integers(0, users, 11)
        pos = (lens[mp][:, None] + np.arange(3)).astype(np.int32)
        Q = dev(rng.standard_normal((11, Hq, 3, dim)), t.bfloat16)
        O = hist.attend(Q, dev(mp.astype(np.int32)), positions=dev(pos))
        q_turned = h.rope(Q.transpose(1, 2).reshape(33, Hq, dim), None, dev(pos.reshape(-1)), hist.freq)[0]
        q_turned = f64(q_turned).reshape(11, 3, Hq, dim).transpose(0, 2, 1, 3)
        want, bound = ref.attend(q_turned, kp, vp, table, lens, mp, None)
        bounded(f64(O), want, bound, t.bfloat16, f"step {step}: candidates")
        # The new tokens themselves, each seeing up to itself; padding rows are left.
        Qn = dev(rng.standard_normal((T, Hq, dim)), t.bfloat16)
        out = t.full_like(Qn, 5.0)
        hist.attend(Qn, tab.rows, positions=tab.positions, causal=True, out=out)
        rows = tab.rows.cpu().numpy()
        p = tab.positions.cpu().numpy()
        qn = f64(h.rope(Qn, None, tab.positions, hist.freq)[0])[:, :, None]
        want, bound = ref.attend(qn, kp, vp, table, lens, rows, p[:, None])
        live = rows >= 0
        bounded(f64(out)[live], want[live][:, :, 0], bound[live][:, :, 0], t.bfloat16, f"step {step}: new tokens")
        assert (out[dev(~live)] == 5).all() and hist.check() == bga.IKBO_OK
    with pytest.raises(ValueError):
        hist.attend(Q, None)
    # A step that the write would refuse leaves the tables where they are.
    k = t.zeros(6, Hkv, dim, dtype=t.bfloat16, device="cuda")
    ones = t.ones(users, dtype=t.int32, device="cuda")
    before = (hist.lens.clone(), hist.state.clone(), hist.table.clone())
    for bad in ((k, k.float()), (k, k[:5]), (k[:, :1], k[:, :1]), (k.half(), k.half()), (k, k.cpu()), (k[..., :32], k[..., :32])):
        with pytest.raises(ValueError):
            hist.append(*bad, ones)
    assert all(t.equal(x, y) for x, y in zip(before, (hist.lens, hist.state, hist.table)))


def test_captured_steps_and_two_graphs_and_streams():
    """A captured step (append and attention) replayed with new inputs against eager steps; two graphs captured on one
    stream replayed on two streams at once; eager calls on two streams at once."""
    t = torch()
    h = H()
    rng = np.random.default_rng(21)

    def make(seed):
        r = np.random.default_rng(seed)
        hist = h.UserHistories(9, 512, 80, 2, 128, rot_dim=128)
        k, v = (dev(r.standard_normal((9 * 100, 2, 128)), t.bfloat16) for _ in range(2))
        hist.append(k, v, t.full((9,), 100, dtype=t.int32, device="cuda"))
        return hist

    def step(hist, k, v, q, counts, out):
        tab = hist.append(k, v, counts)
        hist.attend(q, tab.rows, positions=tab.positions, causal=True, out=out)

    side = t.cuda.Stream()
    sets = []
    for seed in (1, 2):
        hist, eager = make(seed), make(seed)
        k, v = (t.zeros(9, 2, 128, dtype=t.bfloat16, device="cuda") for _ in range(2))
        q, out = (t.zeros(9, 8, 128, dtype=t.bfloat16, device="cuda") for _ in range(2))
        counts = t.ones(9, dtype=t.int32, device="cuda")
        t.cuda.synchronize()
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph, stream=side):
            step(hist, k, v, q, counts, out)
        t.cuda.synchronize()
        sets.append((hist, eager, k, v, q, counts, out, graph))
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for rep in range(6):
        for hist, eager, k, v, q, counts, out, graph in sets:
            for x in (k, v, q):
                x.copy_(dev(rng.standard_normal(tuple(x.shape)), t.bfloat16))
        t.cuda.synchronize()
        for s, (hist, eager, k, v, q, counts, out, graph) in zip(streams, sets):
            with t.cuda.stream(s):
                graph.replay()
        t.cuda.synchronize()
        for hist, eager, k, v, q, counts, out, graph in sets:
            want = t.zeros_like(out)
            step(eager, k, v, q, counts, want)
            assert t.equal(out, want), rep
            assert t.equal(hist.lens, eager.lens) and t.equal(hist.tiles, eager.tiles)
            assert hist.check() == bga.IKBO_OK
    # Eager attention on both streams at once, through the stream argument, many times over.
    wants = [h.kv4_attention(q, hist.tiles, hist.table, hist.lens, None, hist.status) for hist, _, _, _, q, _, _, _ in sets]
    t.cuda.synchronize()
    outs = [[t.empty_like(w) for _ in range(20)] for w in wants]
    for i in range(20):
        for s, o, (hist, _, _, _, q, _, _, _) in zip(streams, outs, sets):
            h.kv4_attention(q, hist.tiles, hist.table, hist.lens, None, hist.status, out=o[i], stream=s)
    t.cuda.synchronize()
    for w, o in zip(wants, outs):
        assert all(t.equal(w, x) for x in o)


def test_attend_on_a_given_stream_behind_a_busy_current_one():
    """Rotary queries of several heads and tokens, and positions that are not contiguous, produced on the stream that the
    call is given while the current stream is busy: the result is that of a call on one stream alone."""
    t = torch()
    h = H()
    rng = np.random.default_rng(23)
    hist = h.UserHistories(5, 256, 20, 2, 64, rot_dim=64)
    k, v = (dev(rng.standard_normal((5 * 150, 2, 64)), t.bfloat16) for _ in range(2))
    hist.append(k, v, t.full((5,), 150, dtype=t.int32, device="cuda"))
    mp = dev((np.arange(70) % 5).astype(np.int32))
    pos = dev(rng.integers(0, 150, (33, 70)).astype(np.int32)).t()
    qs = [dev(rng.standard_normal((70, 4, 33, 64)), t.bfloat16) for _ in range(6)]
    wants = [hist.attend(q, mp, positions=pos) for q in qs]
    big = t.randn(8192, 8192, dtype=t.bfloat16, device="cuda")
    side = t.cuda.Stream()
    t.cuda.synchronize()
    outs = []
    for stream in (side, side.cuda_stream):
        for q, want in zip(qs, wants):
            for _ in range(3):
                big @ big                     # the current stream is busy
            with t.cuda.stream(side):
                mine = q + 0
                at = pos + 0
            outs.append((hist.attend(mine, mp, positions=at, stream=stream), want, mine, at))
            t.full((70 * 33 * 4 * 64,), 7.0, dtype=t.bfloat16, device="cuda")   # takes memory that the current stream has free
    t.cuda.synchronize()
    assert all(t.equal(got, want) for got, want, _, _ in outs)
    assert hist.check() == bga.IKBO_OK


def test_cached_attention_agrees_with_dense_target_attention():
    """FaPlan over the dequantised values and the cached attention over the codes compute the same weights and sums."""
    t = torch()
    h = H()
    rng = np.random.default_rng(22)
    B_u, B_c, heads, Lq, n, dim = 3, 10, 2, 16, 192, 128
    lens = np.full(B_u, n)
    tiles, d_table, table, k, v = history(rng, lens, 3, heads, dim)
    K, V = (dev(np.stack([x[table[u]].transpose(1, 0, 2, 3).reshape(heads, n, dim) for u in range(B_u)]), t.bfloat16) for x in (k, v))
    Q = dev(rng.standard_normal((B_c, heads, Lq, dim)), t.bfloat16)
    mp = np.sort(rng.integers(0, B_u, B_c)).astype(np.int32)
    with bga.FaPlan(B_u, B_c, heads, Lq, n, dim) as plan:
        dense = plan.forward(Q, K, V, dev(mp))
    st = word()
    O = h.kv4_attention(Q, tiles, d_table, dev(lens.astype(np.int32)), dev(mp), st)
    want, bound = ref.attend(f64(Q), k, v, table, lens, mp, None)
    bounded(f64(O), want, bound, t.bfloat16, "cached")
    bounded(f64(dense), want, bound, t.bfloat16, "dense")
