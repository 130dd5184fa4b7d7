"""The cached-history operators on the CPU: refusals at the C ABI before any HIP call, refusals of the binding, the
frequency tables, and the plain forms that the GPU tests compare with (against independent small cases)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import broadcast_gemm_amd as bga
from broadcast_gemm_amd import history
from history_ref import LEVELS, decode, encode, put, put_all, rows_of, tables, turn


# The structures of the C ABI.
_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class _TablesArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("counts", "lens", "lens_out", "block_table", "ring", "state", "state_out", "slots", "positions",
                                    "rows", "starts", "status")]
                + [("table_stride", _i64)] + [(n, _i32) for n in ("B_u", "max_pages", "num_pages", "page_size", "capacity")])


class _RopeArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("q", "k", "q_out", "k_out", "positions", "freq")]
                + [(n, _i64) for n in ("q_token", "q_head", "k_token", "k_head", "q_out_token", "q_out_head", "k_out_token", "k_out_head")]
                + [(n, _i32) for n in ("T", "H_q", "H_k", "head_dim", "rot_dim", "layout", "dtype", "inverse")]
                + [("factor", ctypes.c_float)])


class _RowsArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("k", "v", "slots", "tiles", "status")]
                + [(n, _i64) for n in ("k_token", "k_head", "v_token", "v_head")]
                + [(n, _i32) for n in ("T", "H_kv", "head_dim", "num_pages", "dtype")])


class _AttentionArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("Q", "O", "tiles", "block_table", "lens", "map", "positions", "status", "workspace")]
                + [(n, _i64) for n in ("workspace_bytes", "q_cand", "q_head", "q_query", "o_cand", "o_head", "o_query", "table_stride")]
                + [(n, _i32) for n in ("B_u", "B_c", "H_q", "H_kv", "L_q", "head_dim", "max_pages", "num_pages")]
                + [("scale", ctypes.c_float)])


P = 1 << 20   # a stand-in address: every check below returns before any HIP call
INVALID, UNSUPPORTED, ALIGNMENT = bga.IKBO_ERR_INVALID_ARG, bga.IKBO_ERR_UNSUPPORTED, bga.IKBO_ERR_ALIGNMENT


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(bga.LIB_PATH):
        from broadcast_gemm_amd import build
        build.build()
    return bga.lib()


def call(f, args):
    return f(ctypes.byref(args), None)


def fill(cls, **kw):
    a = cls()
    for name, kind in cls._fields_:
        setattr(a, name, kw.pop(name, P if kind is ctypes.c_void_p else 0))
    assert not kw
    return a


TABLES = dict(table_stride=9, B_u=3, max_pages=9, num_pages=40, page_size=64, capacity=10)


@pytest.mark.parametrize("change, want", [
    (dict(B_u=0), INVALID), (dict(B_u=4097), UNSUPPORTED), (dict(max_pages=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(capacity=-1), INVALID), (dict(table_stride=8), INVALID), (dict(counts=0), INVALID),
    (dict(status=0), INVALID), (dict(slots=0), INVALID), (dict(lens=P + 2), ALIGNMENT), (dict(rows=P + 1), ALIGNMENT),
    (dict(num_pages=1 << 25), UNSUPPORTED), (dict(max_pages=1 << 25, table_stride=1 << 25), UNSUPPORTED)])
def test_tables_refusals(L, change, want):
    assert call(L.ikbo_kv_tables, fill(_TablesArgs, **{**TABLES, **change})) == want
    assert L.ikbo_kv_tables(None, None) == INVALID


ROPE = dict(q_token=512, q_head=128, k_token=256, k_head=128, q_out_token=512, q_out_head=128, k_out_token=256, k_out_head=128,
            q_out=2 * P, k_out=2 * P, T=5, H_q=4, H_k=2, head_dim=128, rot_dim=128, layout=0, dtype=0, inverse=0, factor=1.0)


@pytest.mark.parametrize("change, want", [
    (dict(T=-1), INVALID), (dict(T=0), bga.IKBO_OK), (dict(H_q=0, H_k=0), INVALID), (dict(H_q=-1), INVALID), (dict(rot_dim=7), INVALID),
    (dict(rot_dim=0), INVALID), (dict(rot_dim=130), INVALID), (dict(head_dim=1026), UNSUPPORTED), (dict(layout=2), INVALID),
    (dict(dtype=2), INVALID), (dict(inverse=2), INVALID), (dict(factor=math.inf), INVALID), (dict(factor=math.nan), INVALID),
    (dict(q=0), INVALID), (dict(k_out=0), INVALID), (dict(positions=0), INVALID), (dict(freq=P + 4), ALIGNMENT),
    (dict(q=P + 1), ALIGNMENT), (dict(dtype=1, k=P + 2), ALIGNMENT), (dict(q_out=P, q_out_token=640), INVALID), (dict(H_q=5000), UNSUPPORTED)])
def test_rope_refusals(L, change, want):
    assert call(L.ikbo_rope, fill(_RopeArgs, **{**ROPE, **change})) == want
    assert L.ikbo_rope(None, None) == INVALID


ROWS = dict(k_token=256, k_head=128, v_token=256, v_head=128, T=5, H_kv=2, head_dim=128, num_pages=7, dtype=0)


@pytest.mark.parametrize("change, want", [
    (dict(T=-1), INVALID), (dict(T=0), bga.IKBO_OK), (dict(H_kv=0), INVALID), (dict(num_pages=0), INVALID), (dict(dtype=3), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(num_pages=1 << 25), UNSUPPORTED), (dict(H_kv=5000), UNSUPPORTED), (dict(slots=0), INVALID),
    (dict(tiles=0), INVALID), (dict(status=0), INVALID), (dict(k=P + 8), ALIGNMENT), (dict(tiles=P + 4), ALIGNMENT),
    (dict(k_token=260), ALIGNMENT), (dict(v_head=132), ALIGNMENT)])
def test_rows_refusals(L, change, want):
    args = {**ROWS, **change}
    assert call(L.ikbo_kv4_write, fill(_RowsArgs, **args)) == want
    assert call(L.ikbo_kv4_read, fill(_RowsArgs, **args)) == want
    assert L.ikbo_kv4_write(None, None) == INVALID and L.ikbo_kv4_read(None, None) == INVALID


def test_write_needs_both_tensors(L):
    assert call(L.ikbo_kv4_write, fill(_RowsArgs, **ROWS, v=0)) == INVALID
    assert call(L.ikbo_kv4_read, fill(_RowsArgs, **ROWS, k=0, v=0)) == bga.IKBO_OK


ATTEND = dict(workspace_bytes=1 << 40, q_cand=512, q_head=128, q_query=128, o_cand=512, o_head=128, o_query=128, table_stride=9, B_u=3,
              B_c=6, H_q=4, H_kv=2, L_q=1, head_dim=128, max_pages=9, num_pages=40, scale=0.0)


@pytest.mark.parametrize("change, want", [
    (dict(B_u=0), INVALID), (dict(B_u=4097), UNSUPPORTED), (dict(B_c=-1), INVALID), (dict(B_c=0), bga.IKBO_OK), (dict(H_kv=0), INVALID),
    (dict(H_q=5), INVALID), (dict(H_q=1), INVALID), (dict(L_q=0), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(max_pages=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(num_pages=1 << 25), UNSUPPORTED), (dict(table_stride=8), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(Q=0), INVALID), (dict(O=0), INVALID), (dict(lens=0), INVALID),
    (dict(workspace=0), INVALID), (dict(workspace_bytes=100), INVALID), (dict(map=0), INVALID), (dict(Q=P + 8), ALIGNMENT),
    (dict(q_head=132), ALIGNMENT), (dict(o_query=4), ALIGNMENT), (dict(map=P + 2), ALIGNMENT), (dict(positions=P + 1), ALIGNMENT),
    (dict(B_c=1 << 28, L_q=64), UNSUPPORTED)])
def test_attention_refusals(L, change, want):
    assert call(L.ikbo_kv4_attention, fill(_AttentionArgs, **{**ATTEND, **change})) == want
    assert L.ikbo_kv4_attention(None, None) == INVALID


@pytest.mark.parametrize("change", [dict(o_cand=64 * 128), dict(o_head=256), dict(L_q=2, q_query=128, o_query=256)])
def test_attention_refuses_its_queries_in_another_order(L, change):
    """O may be Q only with Q's strides: a row written elsewhere would be a query not yet read."""
    assert call(L.ikbo_kv4_attention, fill(_AttentionArgs, **{**ATTEND, "O": P, "Q": P, **change})) == INVALID


def test_attention_workspace(L):
    f = L.ikbo_kv4_attention_workspace
    assert f(15, 15, 4, 4, 1, 128, 16) > 0
    assert f(0, 15, 4, 4, 1, 128, 16) == INVALID and f(15, 15, 5, 4, 1, 128, 16) == INVALID
    assert f(15, 15, 4, 4, 1, 80, 16) == UNSUPPORTED


def test_library_is_built_where_its_torch_binding_cannot_be(tmp_path, monkeypatch, capsys):
    """The C ABI needs hipcc alone: without torch it is built and said to be alone, and a host compiler that fails is an
    error that leaves the library linked."""
    import sys

    from broadcast_gemm_amd import build
    try:
        build.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    (tmp_path / "one.cpp").write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "ROOT", str(tmp_path))
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    monkeypatch.setattr(build, "SOURCES", ["one.cpp"])
    monkeypatch.setattr(build, "TORCH_LIB", str(tmp_path / "_ikbo_torch.so"))
    for name, fails in (("a.so", False), ("b.so", True)):
        monkeypatch.setattr(build, "LIB", str(tmp_path / name))
        with monkeypatch.context() as m:
            if fails:
                m.setattr(build, "torch_command", lambda out: [sys.executable, "-c", "import sys; sys.exit('no headers')"])
                with pytest.raises(RuntimeError, match="no headers"):
                    build.build()
            else:
                m.setitem(sys.modules, "torch", None)
                assert build.build() == str(tmp_path / name)
                assert "torch" in capsys.readouterr().err
        assert ctypes.CDLL(str(tmp_path / name)).one() == 1
        assert not (tmp_path / "_ikbo_torch.so").exists()


def test_status_word_refusal(L):
    assert L.ikbo_kv_status(None, None) == INVALID
    for code in (bga.IKBO_ERR_PAGE_RANGE, bga.IKBO_ERR_NO_PAGES, bga.IKBO_ERR_NONFINITE):
        assert bga.status_str(code) != "unknown status"


def test_binding_refuses_host_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    t = torch.zeros(3, 2, 68 * 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        history.kv_tables(i, i, torch.zeros(4, 2, dtype=torch.int32), i, i, 4, i[:1])
    with pytest.raises(ValueError):
        history.rope(x, x, i, torch.ones(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        history.kv4_write(x, x, i, t, i[:1])
    with pytest.raises(ValueError):
        history.kv4_read(i, t, i[:1])
    with pytest.raises(ValueError):
        history.kv4_attention(x, t, torch.zeros(4, 2, dtype=torch.int32), i, None, i[:1])
    with pytest.raises(ValueError):
        history.kv_status(i[:1])
    with pytest.raises(ValueError):
        history.rope(None, None, i, torch.ones(32, dtype=torch.float64))


def test_heads_of_one_tensor_are_told_from_overlap():
    qkv = torch.zeros(6, 8, 64)
    assert history._interleaved(qkv[:, :4], qkv[:, 4:6]) and history._interleaved(qkv[:, 6:], qkv[:, :4])
    assert not history._interleaved(qkv[:, :4], qkv[:, 3:6])
    assert not history._interleaved(qkv[:5], qkv[1:])
    with pytest.raises(ValueError):
        history._distinct("out", torch.zeros(1, 4, 64).expand(6, 4, 64))
    with pytest.raises(ValueError):
        history._distinct("out", torch.zeros(100).as_strided((3, 4, 8), (8, 8, 1)))
    history._distinct("out", qkv.transpose(0, 1))


def test_attention_refuses_an_output_that_meets_its_queries():
    """O may be Q or stand apart from it, also within one tensor; rows of O over other rows of Q are refused."""
    i, st = torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    tiles, table = torch.zeros(3, 2, 68 * 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.int32)
    buf = torch.zeros(5, 8, 6, 64, dtype=torch.bfloat16)
    flat = torch.zeros(5 * 8 * 6 * 64 + 8, dtype=torch.bfloat16)
    wide = torch.zeros(4, 2, 4 * 3 * 64, dtype=torch.bfloat16)

    def attend(Q, out):
        history.kv4_attention(Q, tiles, table, i, None, st, out=out)

    q = buf[:4, :4, :3]
    for out in (buf[1:, :4, :3], buf[:4, 2:6, :3], buf[:4, :4, 2:5], buf[:4, 1:5, 1:4], buf[1:, 3:7, 2:5]):
        with pytest.raises(ValueError, match="overlap"):
            attend(q, out)
    with pytest.raises(ValueError, match="overlap"):
        attend(flat[:4 * 768].view(4, 4, 3, 64), flat[8:8 + 4 * 768].view(4, 4, 3, 64))
    with pytest.raises(ValueError, match="overlap"):
        attend(wide[:, 0].view(4, 4, 3, 64), wide[:, 0].view(4, 3, 4, 64).transpose(1, 2))
    # What stands apart gets as far as the check of the device.
    for a, out in ((q, q), (q, buf[:4, 4:, :3]), (q, buf[:4, :4, 3:]), (buf[:4, 4:, 3:], q), (q, buf[:4, 4:, 2:5]), (q, q.clone()),
                   (wide[:, 0].view(4, 4, 3, 64), wide[:, 1].view(4, 3, 4, 64).transpose(1, 2)), (q[:1], q[:1].as_strided((1, 4, 3, 64), (8, 384, 64, 1)))):
        with pytest.raises(ValueError, match="GPU"):
            attend(a, out)


def test_meeting_tensors_against_their_elements():
    """_meet against the sets of elements: exact, whatever the strides are."""
    rng = np.random.default_rng(4)
    flat = torch.zeros(4000)
    crossed = 0
    for _ in range(3000):
        shapes = rng.integers(1, 5, (2, 3))
        strides = np.cumprod(rng.integers(1, 6, 3))[::-1].copy()
        other = strides if rng.random() < 0.6 else rng.integers(0, 30, 3)
        ta = flat.as_strided(tuple(map(int, shapes[0])), tuple(map(int, strides)), int(rng.integers(0, 200)))
        tb = flat.as_strided(tuple(map(int, shapes[1])), tuple(map(int, other)), int(rng.integers(0, 200)))
        at = [set((x.storage_offset() + sum(np.indices(x.shape)[d] * x.stride(d) for d in range(3))).ravel().tolist()) for x in (ta, tb)]
        meet = bool(at[0] & at[1])
        assert history._meet(ta, tb) == history._meet(tb, ta)
        assert history._meet(ta, tb) == meet
        crossed += not meet and history._spans(ta)[0] < history._spans(tb)[1] and history._spans(tb)[0] < history._spans(ta)[1]
    assert crossed > 200


def test_attend_stays_on_the_stream_it_is_given(monkeypatch):
    """With rotary queries of several heads and tokens, Q has to be copied: the copy, the rotation and the attention all
    belong on the call's stream.  Told on the CPU by a stand-in for entering that stream."""
    import contextlib

    from torch.utils._python_dispatch import TorchDispatchMode

    on, seen = [], []

    @contextlib.contextmanager
    def enter(device, stream):
        on.append(stream)
        yield 0
        on.pop()

    class Watch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            if isinstance(out, torch.Tensor) and out.untyped_storage().data_ptr() not in {a.untyped_storage().data_ptr() for a in args if isinstance(a, torch.Tensor)}:
                seen.append((func.__name__, bool(on)))
            return out

    def rope(q, k, positions, freq, stream=None, **kw):
        seen.append(("rope", bool(on) or stream is not None))
        return q.contiguous(), None

    def attention(Q, *rest, stream=None, **kw):
        seen.append(("attention", bool(on) or stream is not None))
        return Q

    monkeypatch.setattr(history, "_on", enter)
    monkeypatch.setattr(history, "rope", rope)
    monkeypatch.setattr(history, "kv4_attention", attention)
    hist = history.UserHistories(3, 64, 3, 2, 64, rot_dim=64, device="cpu")
    Q = torch.zeros(11, 4, 3, 64, dtype=torch.bfloat16)
    mp, positions = torch.zeros(11, dtype=torch.int32), torch.zeros(3, 11, dtype=torch.int32).t()
    with Watch():
        out = hist.attend(Q, mp, positions=positions, stream="the call's stream")
    assert out.shape == Q.shape and not on
    names = [n for n, _ in seen]
    assert "rope" in names and "attention" in names and len(names) > 2      # the copies were seen
    assert all(there for _, there in seen), seen


# ---- frequencies ---------------------------------------------------------------------------


def test_frequencies_plain_linear_theta():
    f, a = history.rope_frequencies(64, 500.0, device="cpu")
    assert a == 1.0 and f.dtype == torch.float64
    for i in range(32):
        assert float(f[i]) == pytest.approx(500.0 ** (-2 * i / 64), rel=1e-14)
    g, _ = history.rope_frequencies(64, 500.0, {"kind": "linear", "factor": 4}, device="cpu")
    assert torch.allclose(g * 4, f, rtol=1e-15)
    g, _ = history.rope_frequencies(64, 500.0, {"kind": "theta", "factor": 4}, device="cpu")
    assert float(g[0]) == 1.0 and float(g[31]) == pytest.approx(float(f[31]) / 4, rel=1e-12)


def test_frequencies_ramps():
    how = dict(factor=8, context=8192, low=1, high=4)
    f, _ = history.rope_frequencies(128, 1e4, device="cpu")
    g, a = history.rope_frequencies(128, 1e4, {"kind": "turns", **how}, device="cpu")
    assert a == 1.0
    for x, y in zip(f.tolist(), g.tolist()):
        turns = 8192 * x / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1) / 3))
        assert y == pytest.approx(x * keep + x / 8 * (1 - keep), rel=1e-13)
    how.update(low=1, high=32)
    g, a = history.rope_frequencies(128, 1e4, {"kind": "pairs", **how}, device="cpu")
    assert a == pytest.approx(0.1 * math.log(8) + 1)
    ratio = (g / f).tolist()
    assert ratio[0] == 1.0 and ratio[-1] == pytest.approx(1 / 8) and all(x >= y - 1e-12 for x, y in zip(ratio, ratio[1:]))
    turns = [8192 * x / (2 * math.pi) for x in f.tolist()]
    assert all(r == pytest.approx(1.0) for r, t in zip(ratio, turns) if t > 40) and all(r == pytest.approx(1 / 8) for r, t in zip(ratio, turns) if t < 0.8)
    assert history.rope_frequencies(128, 1e4, {"kind": "pairs", "attention": 1.5, **how}, device="cpu")[1] == 1.5


@pytest.mark.parametrize("rot, scaling", [(7, None), (0, None), (64, {"kind": "linear", "factor": 0}), (64, {"kind": "other", "factor": 2}),
                                          (2, {"kind": "theta", "factor": 2}), (64, {"kind": "turns", "factor": 2, "context": 8, "low": 4, "high": 1})])
def test_frequencies_refusals(rot, scaling):
    with pytest.raises(ValueError):
        history.rope_frequencies(rot, 1e4, scaling, device="cpu")


@pytest.mark.parametrize("cast", ["bfloat16", "half", "float", "double", "to", "type", "meta"])
def test_rope_frequencies_survive_casts_of_their_module(cast):
    """A model that holds IkboRope is cast as any other: its parameters change, the frequencies stay float64 to the bit."""
    from broadcast_gemm_amd.autograd import IkboRope
    want, _ = history.rope_frequencies(64, 500.0, device="cpu")
    rope = IkboRope(64, theta=500.0)
    model = torch.nn.Sequential(torch.nn.Linear(2, 2), rope)
    if cast == "to":
        model.to(torch.bfloat16)
    elif cast == "type":
        model.type(torch.float16)
    elif cast == "meta":
        model.to("meta", torch.bfloat16)
        assert rope.freq.dtype == torch.float64 and rope.freq.device.type == "meta" and model[0].weight.dtype == torch.bfloat16
        return
    else:
        getattr(model, cast)()
    assert model[0].weight.dtype == {"float": torch.float32, "double": torch.float64, "half": torch.float16, "type": torch.float16}.get(cast, torch.bfloat16)
    model.double()
    assert rope.freq.dtype == torch.float64 and torch.equal(rope.freq, want)
    assert dict(rope.named_buffers())["freq"] is rope.freq and not rope.state_dict()


# ---- the plain forms -----------------------------------------------------------------------


def test_plain_codes():
    x = np.zeros((1, 32))
    x[0, :10] = [6, 5, -5, 0.25, -0.75, 1.25, 1.75, 2.5, 3.5, 0.26]
    c, s = encode(x)
    assert s[0, 0] == 127
    assert decode(c, s)[0, :10].tolist() == [6, 4, -4, 0, -1, 1, 2, 2, 4, 0.5]
    assert encode(x * 1.0001)[1][0, 0] == 128                       # 6.0006 no longer fits the scale 1
    assert encode(np.zeros((1, 32)))[1][0, 0] == 2
    rng = np.random.default_rng(0)
    y = rng.standard_normal((50, 64)) * np.exp(3 * rng.standard_normal((50, 1)))
    z = decode(*encode(y))
    # Levels are at most 2 apart at the scale, and the largest magnitude is over 3: within half a gap of 1.
    top = np.abs(y.reshape(50, 2, 32)).max(-1, keepdims=True)
    assert (np.abs(z - y).reshape(50, 2, 32) <= top / 3 * 1.0000001).all()
    assert len(LEVELS) == 8


@pytest.mark.parametrize("dim", [64, 128])
def test_plain_rows_at_once(dim):
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 150, 3, dim)) * np.exp(rng.standard_normal((2, 150, 3, 1)))
    slots = rng.permutation(256)[:150].astype(np.int32)
    slots[[4, 90]] = -1
    one, all_ = (np.full((4, 3, 68 * dim), 0x5A, np.uint8) for _ in range(2))
    put(one, k, v, slots)
    put_all(all_, k, v, slots)
    assert np.array_equal(one, all_)
    live = slots >= 0
    for x, y in zip((k, v), rows_of(all_)):
        assert np.array_equal(y[slots[live] // 64, :, slots[live] % 64], decode(*encode(x[live])))


def test_plain_turn_keeps_lengths_and_inverts():
    rng = np.random.default_rng(1)
    x, pos, f = rng.standard_normal((5, 2, 10)), np.array([0, 1, 7, 100, 10 ** 6]), np.array([1.0, 0.3, 0.01])
    for layout in ("half", "interleaved"):
        y, _ = turn(x, pos, f, layout)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[0], x[0]) and np.array_equal(y[..., 6:], x[..., 6:])
        assert np.allclose(turn(y, pos, f, layout, inverse=True)[0], x)


def test_plain_tables():
    table, ring = np.full((3, 4), -1, np.int32), np.arange(10, 18, dtype=np.int32)
    got = tables([3, 0, 5], [0, 0, 0], table, ring, 6, 8, 10, P=4)
    assert got[0].tolist() == [64, 65, 66, 68, 69, 70, 71, 40, -1, -1] and got[5:] == (1, 5)
    got = tables([-1, 1, 1], got[4], table, ring, got[5], got[6], 2, P=4)
    assert got[0].tolist() == [44, 41] and got[4].tolist() == [0, 1, 6] and got[5:] == (2, 5) and ring[6] == 16
    assert tables([1, 1, 1], got[4], table, ring, got[5], got[6], 2, P=4) is None
