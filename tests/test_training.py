"""Attention's training and dropout on the CPU: refusals at the C ABI before any HIP call, the workspace's bounds, the
generator, and the plain form that the GPU tests compare with (against differences)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import broadcast_gemm_amd as bga
import training_ref as ref
from broadcast_gemm_amd.autograd import IkboAttention, IkboDropout, IkboLce

_vp, _i32, _i64, _f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double


class _AttentionArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("Q", "K", "V", "O", "lse", "dO", "dQ", "dK", "dV", "map", "lens", "positions", "rng", "status", "workspace")]
                + [(n, _i64) for n in ("workspace_bytes", "q_cand", "q_head", "q_query", "k_user", "k_head", "k_token", "v_user", "v_head",
                                       "v_token", "o_cand", "o_head", "o_query", "do_cand", "do_head", "do_query", "dq_cand", "dq_head",
                                       "dq_query", "dk_user", "dk_head", "dk_token", "dv_user", "dv_head", "dv_token")]
                + [("dropout", _f64)] + [(n, _i32) for n in ("B_u", "B_c", "H_q", "H_kv", "L_q", "L_kv", "head_dim")]
                + [("scale", ctypes.c_float)])


class _DropoutArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("x", "residual", "y", "rng")] + [("n", _i64), ("p", _f64), ("dtype", _i32)]


P = 1 << 20   # a stand-in address: every check below returns before any HIP call
OK, INVALID, UNSUPPORTED, ALIGNMENT = bga.IKBO_OK, bga.IKBO_ERR_INVALID_ARG, bga.IKBO_ERR_UNSUPPORTED, bga.IKBO_ERR_ALIGNMENT


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(bga.LIB_PATH):
        from broadcast_gemm_amd import build
        build.build()
    return bga.lib()


def fill(cls, **kw):
    a = cls()
    for name, kind in cls._fields_:
        setattr(a, name, kw.pop(name, P if kind is _vp else 0))
    assert not kw
    return a


ATTEND = dict(workspace_bytes=1 << 40, B_u=3, B_c=5, H_q=4, H_kv=2, L_q=2, L_kv=100, head_dim=128, q_cand=1024, q_head=256, q_query=128,
              k_user=25600, k_head=12800, k_token=128, v_user=25600, v_head=12800, v_token=128, o_cand=1024, o_head=256, o_query=128)

COMMON = [
    (dict(B_u=0), INVALID), (dict(B_c=-1), INVALID), (dict(H_q=3), INVALID), (dict(H_q=1), INVALID), (dict(H_kv=0), INVALID), (dict(L_q=0), INVALID),
    (dict(L_kv=0), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(B_u=4097), UNSUPPORTED),
    (dict(H_q=8192, H_kv=2), UNSUPPORTED), (dict(B_c=1 << 30), UNSUPPORTED), (dict(B_c=1 << 20, L_q=1 << 12), UNSUPPORTED),
    (dict(L_kv=(1 << 31) - 1), UNSUPPORTED), (dict(B_u=4096, H_q=4096, H_kv=4096, L_kv=1000), UNSUPPORTED),
    (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(dropout=-0.1), INVALID), (dict(dropout=1.0), INVALID), (dict(dropout=math.nan), INVALID), (dict(dropout=0.001), INVALID),
    (dict(dropout=0.999), INVALID), (dict(dropout=0.5, rng=0), INVALID), (dict(q_head=-256), INVALID), (dict(q_query=132), ALIGNMENT),
    (dict(k_token=4), ALIGNMENT), (dict(o_cand=12), ALIGNMENT), (dict(Q=P + 8), ALIGNMENT), (dict(V=P + 2), ALIGNMENT), (dict(O=P + 4), ALIGNMENT),
    (dict(lse=P + 2), ALIGNMENT), (dict(map=P + 1), ALIGNMENT), (dict(lens=P + 2), ALIGNMENT), (dict(positions=P + 2), ALIGNMENT),
    (dict(rng=P + 4), ALIGNMENT), (dict(workspace=P + 8), ALIGNMENT), (dict(status=0), INVALID), (dict(workspace=0), INVALID),
    (dict(workspace_bytes=255), INVALID), (dict(Q=0), INVALID), (dict(K=0), INVALID), (dict(V=0), INVALID), (dict(O=0), INVALID),
    (dict(lse=0), INVALID), (dict(map=0), INVALID), (dict(k_token=(1 << 24) + 8), UNSUPPORTED), (dict(v_token=(1 << 24) + 8), UNSUPPORTED)]


@pytest.mark.parametrize("change, want", COMMON + [(dict(B_c=0, Q=0, O=0, map=0), OK)])
def test_forward_refusals(L, change, want):
    assert L.ikbo_attention_forward(ctypes.byref(fill(_AttentionArgs, **{**ATTEND, **change})), None) == want
    assert L.ikbo_attention_forward(None, None) == INVALID


@pytest.mark.parametrize("change, want", COMMON + [
    (dict(dO=0), INVALID), (dict(dQ=0), INVALID), (dict(dK=0), INVALID), (dict(dV=0), INVALID), (dict(B_c=0, dV=0), INVALID),
    (dict(dO=P + 8), ALIGNMENT), (dict(dK=P + 8), ALIGNMENT), (dict(do_head=4), ALIGNMENT), (dict(dv_token=-8), INVALID)])
def test_backward_refusals(L, change, want):
    assert L.ikbo_attention_backward(ctypes.byref(fill(_AttentionArgs, **{**ATTEND, **change})), None) == want
    assert L.ikbo_attention_backward(None, None) == INVALID


@pytest.mark.parametrize("change", [dict(K=0), dict(V=0), dict(K=0, V=0)])
def test_gradients_without_candidates_need_the_users_keys(L, change):
    """dK and dV are written all the same, by a kernel that is given K and V."""
    assert L.ikbo_attention_backward(ctypes.byref(fill(_AttentionArgs, **{**ATTEND, "B_c": 0, **change})), None) == INVALID


@pytest.mark.parametrize("change, want", [
    (dict(n=-1), INVALID), (dict(n=0, x=0), OK), (dict(p=-0.1), INVALID), (dict(p=1.0), INVALID), (dict(p=math.nan), INVALID), (dict(p=1e-6), INVALID),
    (dict(dtype=2), INVALID), (dict(x=0), INVALID), (dict(y=0), INVALID), (dict(rng=0), INVALID), (dict(x=P + 1), ALIGNMENT),
    (dict(dtype=1, y=P + 2), ALIGNMENT), (dict(residual=P + 1), ALIGNMENT), (dict(rng=P + 4), ALIGNMENT)])
def test_dropout_refusals(L, change, want):
    assert L.ikbo_dropout(ctypes.byref(fill(_DropoutArgs, **{**dict(n=100, p=0.5), **change})), None) == want
    assert L.ikbo_dropout(None, None) == INVALID


def test_workspace(L):
    f = L.ikbo_attention_workspace
    assert f(15, 1024, 4, 4, 64, 1024, 128, 0) > 0 and f(15, 0, 4, 4, 64, 1024, 128, 1) > 0
    assert f(0, 15, 4, 4, 1, 100, 128, 0) == INVALID and f(15, 15, 5, 4, 1, 100, 128, 0) == INVALID and f(15, 15, 4, 4, 1, 100, 80, 1) == UNSUPPORTED
    # Partial results stay within some hundred MB, whatever the shape.
    for shape in ((1, 8, 8, 1, 1, 1 << 20, 128), (4096, 100000, 8, 8, 1, 512, 64), (1, 500000, 8, 8, 1, 2000, 128), (2, 20000, 16, 4, 64, 64, 128)):
        assert f(*shape, 1) < 4 * shape[1] * shape[2] * shape[4] + (1 << 30), shape


@pytest.mark.parametrize("B_c, L_kv, dim", [(1 << 26, 1 << 22, 64), (1 << 26, (1 << 22) - 1000, 64), (1 << 26, 3 << 21, 64), (1 << 26, 1 << 23, 64),
                                            (1 << 26, 1 << 24, 128), (1 << 28, 1 << 24, 64), (45_000_000, 50_000, 64)])
def test_workspace_of_many_rows_over_many_keys(L, B_c, L_kv, dim):
    """One user's rows are not cut however many keys there are: 4 bytes of order, a quarter of a table entry and 48 bytes of notes a row."""
    assert 52 * B_c < L.ikbo_attention_workspace(1, B_c, 1, 1, 1, L_kv, dim, 1) < 53 * B_c


def test_generator_gives_the_published_numbers():
    """Known answers of Philox4x32 for a counter and key of zeros, with 7 rounds and 10."""
    assert [hex(x) for x in ref.philox(np.zeros(4, np.uint64), 0)] == ["0x5f6fb709", "0xd893f64", "0x4f121f81", "0x4f730a48"]
    assert [hex(x) for x in ref.philox(np.zeros(4, np.uint64), 0, 10)] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]


def test_shares_that_stay():
    """Of 2^19 weights and elements, the share kept is that of the steps, within five standard deviations."""
    for kept, share in ((ref.weights_kept(np.arange(512), 3, 1024, 0.1, (7, 9)), 1 - 26 / 256), (ref.elements_kept(1 << 19, 0.1, (7, 9)), 1 - 6554 / 65536)):
        assert abs(kept.mean() - share) < 5 * math.sqrt(share * (1 - share) / kept.size)
    a, b, c = (ref.weights_kept(np.arange(64), h, 640, 0.5, (7, o)) for h, o in ((0, 0), (1, 0), (0, 1)))
    assert 0.45 < (a == b).mean() < 0.55 and 0.45 < (a == c).mean() < 0.55


@pytest.mark.parametrize("dropout", [0.0, 0.3])
def test_plain_gradients_are_those_of_differences(dropout):
    rng = np.random.default_rng(3)
    Q, K, V = rng.normal(size=(4, 4, 2, 8)), rng.normal(size=(2, 2, 9, 8)), rng.normal(size=(2, 2, 9, 8))
    how = dict(mp=np.array([0, 1, -1, 0]), lens=np.array([9, 5]), positions=np.array([[8, 3], [2, -1], [4, 4], [0, 20]]), dropout=dropout, rng=(5, 6))
    dO = rng.normal(size=Q.shape)
    want = ref.attention(Q, K, V, dO=dO, **how)
    for name, x in (("dQ", Q), ("dK", K), ("dV", V)):
        for _ in range(40):
            i = tuple(rng.integers(0, n) for n in x.shape)
            at = x[i]
            side = []
            for step in (1e-5, -1e-5):
                x[i] = at + step
                side.append((ref.attention(Q, K, V, **how)["O"] * dO).sum())
            x[i] = at
            # Central differences of step 1e-5: third derivatives times 1e-10, and 2^-52 of a sum of about 30 over 2e-5.
            assert abs((side[0] - side[1]) / 2e-5 - want[name][i]) < 1e-7, (name, i)


def test_plain_form_of_known_cases():
    V = np.arange(24.0).reshape(1, 1, 3, 8)
    Q, K = np.ones((3, 1, 2, 8)), np.zeros((1, 1, 3, 8))
    x = ref.attention(Q, K, V, mp=[0, -1, 0], positions=np.array([[1, 0], [1, 1], [-1, 5]]), dO=np.ones_like(Q))
    assert np.allclose(x["O"][0, 0], [(V[0, 0, 0] + V[0, 0, 1]) / 2, V[0, 0, 0]]) and np.allclose(x["lse"][0, 0], [math.log(2), 0])
    assert (x["O"][1] == 0).all() and np.isneginf(x["lse"][1]).all() and (x["O"][2, 0, 0] == 0).all() and np.isneginf(x["lse"][2, 0, 0])
    assert np.allclose(x["O"][2, 0, 1], V[0, 0].mean(0)) and (x["dQ"] == 0).all()
    assert np.allclose(x["dV"][0, 0, :, 0], [0.5 + 1 + 1 / 3, 0.5 + 1 / 3, 1 / 3])


def test_modules_refuse_probabilities_and_keep_their_counters():
    for p in (-0.1, 1.0, 1.5, math.nan, 1e-3):
        with pytest.raises(ValueError):
            IkboAttention(dropout=p)
    for p in (-0.1, 1.0, 1e-6):
        with pytest.raises(ValueError):
            IkboDropout(p)
    a, b = IkboAttention(dropout=0.1), IkboAttention(dropout=0.1)
    assert a.rng.tolist() != b.rng.tolist() and a.rng.dtype == torch.int64
    a.bfloat16()
    assert a.rng.dtype == torch.int64 and a.status.dtype == torch.int32
    first = a._draw()
    assert first.tolist() == [a.rng[0], 0] and a.rng[1] == 1
    b.load_state_dict(a.state_dict())
    assert b.rng.tolist() == a.rng.tolist() and "status" not in a.state_dict()
    assert IkboLce(8, 8, 4, 32).drop is None and IkboLce(8, 8, 4, 32, dropout=0.1).drop.p == 0.1


@pytest.mark.parametrize("reentrant", [False, True])
def test_a_forward_pass_that_is_run_again_draws_the_same_numbers(reentrant):
    from torch.utils.checkpoint import checkpoint
    drop, seeded, drawn = IkboDropout(0.5), IkboDropout(0.5, seed=3), []

    def layer(module, x):
        drawn.append(module._numbers(x.device).tolist())
        return x * x

    x = torch.ones(3, requires_grad=True)
    y = checkpoint(layer, drop, x, use_reentrant=reentrant) + checkpoint(layer, drop, 2 * x, use_reentrant=reentrant)
    y.sum().backward()
    assert len(drawn) == 4 and drawn[0] != drawn[1] and sorted(drawn[:2]) == sorted(drawn[2:])
    # A counter of the module's own would have moved on: refused, in the second pass.
    y = checkpoint(layer, seeded, x, use_reentrant=reentrant).sum()
    with pytest.raises(RuntimeError, match="seed"):
        y.backward()
    assert drawn[4:] == [[3, 0]] and seeded.rng.tolist() == [3, 1]


def test_dropout_in_evaluation_is_the_sum():
    x, r = torch.randn(5), torch.randn(5)
    d = IkboDropout(0.5).eval()
    assert d(x) is x and torch.equal(d(x, r), r + x)


def test_tensors_on_the_host_are_refused():
    from broadcast_gemm_amd import training
    x = torch.zeros(2, 1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        training.attention(x, x, x, torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        training.dropout(x, 0.1, torch.zeros(2, dtype=torch.int64))


def test_numbers_of_64_bits_are_not_wrapped():
    from broadcast_gemm_amd.autograd import _int32
    t = torch.tensor([[-1 << 63, -(1 << 32) - 1, -1], [1 << 32, (1 << 63) - 1, 7]])
    assert _int32(t).tolist() == [[-1 << 31, -1 << 31, -1], [(1 << 31) - 1, (1 << 31) - 1, 7]] and _int32(t.t()).is_contiguous()
    assert _int32(t.to(torch.int32)).dtype == torch.int32 and _int32(torch.tensor([3, 250], dtype=torch.uint8)).tolist() == [3, 250]


def test_status_is_the_modules_own():
    """It moves with the module and is neither cast, saved, nor among the buffers that a wrapper broadcasts between ranks."""
    import copy
    m = torch.nn.Sequential(IkboAttention(dropout=0.1), torch.nn.Linear(2, 2))
    assert set(dict(m.named_buffers())) == {"0.rng"} and "0.status" not in m.state_dict()
    m[0].status[0] = 2
    assert m.bfloat16().double()[0].status.tolist() == [2] and m[0].status.dtype == torch.int32
    other = copy.deepcopy(m)
    other[0].status.zero_()
    assert m[0].status.tolist() == [2]
    assert m.to("meta")[0].status.is_meta and m.to_empty(device="cpu")[0].status.tolist() == [0]
