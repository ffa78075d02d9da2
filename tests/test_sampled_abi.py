"""Argument checks of tree_positions, qkv_rope, kv_append and tree_verify_sampled: refused on the
host, before any CUDA call, with the status and reason of the C ABI."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def w12():
    import lossless_bit_weights_gb300 as m
    m.lib()
    return m


V = ctypes.c_void_p
X, POS, Q, K, U, SLOT, ST = (V(i << 20) for i in range(1, 8))


def form(w12, **kw):
    f = dict(q_norm=256, k_norm=256, inv_freq=256, eps=1e-6, rot_scale=1.0, n_q_heads=4, n_heads=2, head_dim=128,
             rot_dim=128, interleaved=0)
    f.update(kw)
    return ctypes.byref(w12.qkv_form(*[f[n] for n, _ in w12.qkv_form._fields_]))


def cache(w12, **kw):
    c = dict(k=1 << 30, v=1 << 31, n_layers=2, n_blocks=8, layer_stride=8 * 16 * 2 * 128, block_stride=16 * 2 * 128,
             token_stride=2 * 128, head_stride=128, block_size=16, n_heads=2, head_dim=128)
    c.update(kw)
    return ctypes.byref(w12.kv_cache(*[c[n] for n, _ in w12.kv_cache._fields_]))


def rope(w12, f=None, **kw):
    a = dict(x=X, bf16=0, xs=1024, M=4, pos=POS, q=Q, qs=512, k=K, ks=256, v=U, vs=256)
    a.update(kw)
    a = list(a.values())
    return w12.lib().qkv_rope(*a[:4], form(w12) if f is None else f, *a[4:], None)


def append(w12, f=None, c=None, **kw):
    a = dict(x=X, bf16=0, xs=1024, M=4, pos=POS, layer=0, slot=SLOT, q=Q, qs=512, k=K, ks=256, v=U, vs=256, status=ST)
    a.update(kw)
    a = list(a.values())
    return w12.lib().kv_append(*a[:4], form(w12) if f is None else f, a[4], cache(w12) if c is None else c, *a[5:], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(pos=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(M=0), 2), (dict(M=1 << 31), 2), (dict(xs=1023), 2), (dict(qs=504), 2), (dict(ks=128), 2), (dict(vs=0), 2),
    (dict(x=V((1 << 20) + 8)), 1), (dict(xs=1028), 1), (dict(qs=516), 1), (dict(k=V((4 << 20) + 2)), 1),
    (dict(q=X), 1), (dict(q=X, bf16=1), 1),                       # q over float rows; q's stride is not the rows'
    (dict(k=Q), 1), (dict(v=V((3 << 20) + 256)), 1), (dict(pos=Q), 1)])
def test_rope_arguments(w12, kw, status):
    assert rope(w12, **kw) == status
    assert w12.lib().w12_last_error().startswith(b"qkv_rope")


@pytest.mark.parametrize("kw,status", [
    (dict(n_q_heads=0), 2), (dict(n_heads=0), 2), (dict(n_q_heads=70000), 2), (dict(head_dim=0), 2), (dict(head_dim=4), 2),
    (dict(head_dim=12), 2), (dict(head_dim=264), 2), (dict(rot_dim=-8), 2), (dict(rot_dim=4), 2), (dict(rot_dim=136), 2),
    (dict(inv_freq=None), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(rot_scale=float("inf")), 1),
    (dict(rot_scale=float("nan")), 1)])
def test_forms(w12, kw, status):
    assert rope(w12, form(w12, **kw)) == status
    assert append(w12, form(w12, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(pos=None), 1), (dict(slot=None), 1), (dict(status=None), 1), (dict(layer=2), 2),
    (dict(layer=-1), 2), (dict(q=V(1 << 30)), 1), (dict(x=V((1 << 31) + 4096)), 1), (dict(slot=V((1 << 30) + 64)), 1),
    (dict(slot=Q), 1), (dict(M=0), 2)])
def test_append_arguments(w12, kw, status):
    assert append(w12, **kw) == status
    assert w12.lib().w12_last_error().startswith(b"kv_append")


def test_append_cache(w12):
    assert w12.lib().kv_append(X, 0, 1024, 4, form(w12), POS, None, 0, SLOT, Q, 512, K, 256, U, 256, ST, None) == 1
    assert append(w12, c=cache(w12, n_heads=1)) == 2 and append(w12, c=cache(w12, head_dim=64)) == 2
    assert append(w12, c=cache(w12, token_stride=12)) == 1 and append(w12, c=cache(w12, block_size=0)) == 2
    assert w12.lib().kv_append(X, 0, 1024, 4, None, POS, cache(w12), 0, SLOT, Q, 512, K, 256, U, 256, ST, None) == 1


def test_position_arguments(w12):
    def call(len=X, parent=K, off=Q, n_req=2, rows=4, pos=POS, status=ST):
        return w12.lib().tree_positions(len, parent, off, n_req, rows, pos, status, None)

    assert call(len=None) == 1 and call(pos=None) == 1 and call(status=None) == 1 and call(off=None) == 1
    assert call(n_req=0) == 2 and call(n_req=70000) == 2 and call(rows=0) == 2 and call(rows=1 << 31) == 2
    assert call(pos=X) == 1 and call(pos=K) == 1 and call(pos=V((3 << 20) + 8)) == 1 and call(status=POS) == 1


def sampled(w12, **kw):
    a = dict(logits=V(1 << 40), stride=100, M=4, V=100, probs=None, ps=0, parent=X, draft=POS, off=None, n_req=1, u=Q, ub=K,
             T=None, plen=U, nodes=SLOT, bonus=V(8 << 20), status=ST, ws=V(1 << 36), wsb=1 << 20)
    a.update(kw)
    return w12.lib().tree_verify_sampled(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    *[({name: None}, 1) for name in ("logits", "parent", "draft", "u", "ub", "plen", "nodes", "bonus", "status", "ws")],
    (dict(M=0), 2), (dict(M=65535 * 1024 + 1), 2), (dict(V=0), 2), (dict(V=(1 << 31) - 15, stride=1 << 31), 2),
    (dict(stride=99), 2),
    (dict(probs=V(1 << 41), ps=99), 2), (dict(n_req=0), 2), (dict(n_req=70000), 2), (dict(n_req=2), 1),
    (dict(ws=V((1 << 36) + 8)), 1), (dict(wsb=0), 3),
    (dict(plen=Q), 1), (dict(nodes=POS), 1), (dict(bonus=U), 1), (dict(status=SLOT), 1), (dict(ws=V(1 << 40)), 1),
    (dict(bonus=V((1 << 40) + 1596)), 1), (dict(T=V(8 << 20)), 1), (dict(probs=V(1 << 36), ps=100), 1)])
def test_sampled_arguments(w12, kw, status):
    assert sampled(w12, **kw) == status
    assert w12.lib().w12_last_error().startswith(b"tree_verify_sampled")


def test_sampled_workspace(w12):
    size = w12.lib().tree_verify_sampled_workspace_size
    assert sampled(w12, wsb=size(4, 100) - 1) == 3
    assert size(0, 10) == 0 and size(10, 0) == 0
    assert size(1, 1) == 32 and size(1, 1021) == 32 and size(1, 1022) == 48 and size(192, 151936) == 16 + 192 * 149 * 16


def test_binding_refusals(w12):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 1024)
    with pytest.raises(ValueError):
        w12.tree_verify_sampled(x, x, x, x, x)               # not on a GPU
    with pytest.raises(ValueError):
        w12.tree_positions(torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        w12.QKVForm(4, 2, 128, q_norm=torch.zeros(128))
    with pytest.raises(ValueError):
        w12.QKVForm(4, 2, 128, inv_freq=torch.zeros(64))
    f = w12.QKVForm(4, 2, 128)
    assert f.width == 1024
    with pytest.raises(TypeError):
        w12.qkv_rope(x.half(), f, None)
    with pytest.raises(ValueError):
        w12.qkv_rope(x, f, None)
