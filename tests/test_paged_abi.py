"""Argument checks of the paged-cache and logit-rule calls: refused on the host, before any
CUDA call, with the status and reason of the C ABI."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def w12():
    import lossless_bit_weights_gb300 as m
    m.lib()
    return m


P = ctypes.c_void_p(256)


def cache(w12, **kw):
    c = dict(k=256, v=256, n_layers=2, n_blocks=8, layer_stride=8 * 16 * 2 * 128, block_stride=16 * 2 * 128,
             token_stride=2 * 128, head_stride=128, block_size=16, n_heads=2, head_dim=128)
    c.update(kw)
    return ctypes.byref(w12.kv_cache(*[c[n] for n, _ in w12.kv_cache._fields_]))


def attn(w12, c=None, **kw):
    a = dict(q=P, qs=512, k=P, ks=256, v=P, vs=256, M=4, hq=4, layer=0, table=P, ts=3, tw=3, lens=P, parent=P, off=None,
             n_req=1, scale=0.1, out=P, status=P, ws=P, wsb=1 << 40)
    a.update(kw)
    return w12.lib().tree_attn(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["M"], a["hq"],
                               cache(w12) if c is None else c, a["layer"], a["table"], a["ts"], a["tw"], a["lens"],
                               a["parent"], a["off"], a["n_req"], a["scale"], a["out"], a["status"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(parent=None), 1), (dict(out=None), 1),
    (dict(status=None), 1), (dict(ws=None), 1), (dict(q=ctypes.c_void_p(264)), 1), (dict(qs=516), 1), (dict(ks=-8), 1),
    (dict(M=0), 2), (dict(M=1 << 31), 2), (dict(hq=3), 2), (dict(hq=0), 2), (dict(n_req=0), 2), (dict(n_req=70000), 2),
    (dict(n_req=2), 1), (dict(ts=2), 2), (dict(tw=0), 2), (dict(layer=2), 2), (dict(layer=-1), 2),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(wsb=0), 3)])
def test_attention_arguments(w12, kw, status):
    assert attn(w12, **kw) == status
    assert w12.lib().w12_last_error().startswith(b"tree_attn")


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=264), 1), (dict(token_stride=12), 1), (dict(block_stride=-8), 1), (dict(block_size=0), 2),
    (dict(n_blocks=0), 2), (dict(n_blocks=1 << 31), 2), (dict(n_heads=0), 2), (dict(head_dim=96), 2)])
def test_cache_descriptors(w12, kw, status):
    assert attn(w12, cache(w12, **kw)) == status


def test_write_arguments(w12):
    lib = w12.lib()

    def call(c=None, layer=0, layers=1, k=P, kl=0, kr=256, v=P, vl=0, vr=256, rows=4, slot=P, src=None, n=4, status=P):
        return lib.kv_write(cache(w12) if c is None else c, layer, layers, k, kl, kr, v, vl, vr, rows, slot, src, n, status,
                            None)

    assert call(k=None) == 1 and call(slot=None) == 1 and call(status=None) == 1
    assert call(v=ctypes.c_void_p(264)) == 1 and call(kr=4) == 1 and call(vl=-8) == 1
    assert call(layer=2) == 2 and call(layer=1, layers=2) == 2 and call(layers=0) == 2
    assert call(n=0) == 2 and call(rows=0) == 2
    assert call(cache(w12, head_dim=12)) == 2 and call(cache(w12, head_dim=2048)) == 2
    assert lib.kv_write(None, 0, 1, P, 0, 8, P, 0, 8, 1, P, None, 1, P, None) == 1


def test_slot_arguments(w12):
    def call(**kw):
        a = dict(len=P, add=P, extra=0, n_req=2, table=P, ts=4, tw=4, pool=P, nb=8, pos=P, bs=16, path=None, off=None,
                 nodes=0, cap=8, slot=P, src=P, new=ctypes.c_void_p(512), pos_out=ctypes.c_void_p(512), total=P, status=P)
        a.update(kw)
        return w12.lib().kv_slots(*a.values(), None)

    for name in ("len", "add", "table", "pool", "pos", "slot", "src", "new", "pos_out", "total", "status"):
        assert call(**{name: None}) == 1, name
    assert call(pos_out=P) == 1 and call(new=P) == 1          # results may not be the inputs
    assert call(n_req=0) == 2 and call(n_req=4097) == 2 and call(bs=0) == 2 and call(ts=3) == 2 and call(tw=0) == 2
    assert call(nb=0) == 2 and call(cap=0) == 2 and call(cap=1 << 31) == 2
    assert call(path=P, nodes=0, off=P) == 2 and call(path=P, nodes=4) == 1


def test_rule_arguments(w12):
    lib = w12.lib()

    def rules(**kw):
        r = w12.logit_rules()
        for k, v in kw.items():
            setattr(r, k, v)
        return ctypes.byref(r)

    def process(r=None, logits=P, stride=100, M=4, V=100, parent=P, draft=P, off=None, n_req=1, out=P, os=100, status=P):
        return lib.logits_process(logits, stride, M, V, rules() if r is None else r, parent, draft, off, n_req, out, os,
                                  status, None)

    assert process(logits=None) == 1 and process(out=None) == 1 and process(status=None) == 1
    assert process(draft=None) == 1 and process(n_req=2) == 1
    assert process(M=0) == 2 and process(V=0) == 2 and process(stride=99) == 2 and process(os=99) == 2
    assert process(n_req=0, off=P) == 2 and process(n_req=70000, off=P) == 2
    assert process(rules(hist=256)) == 1                      # no lengths
    assert process(rules(bias_off=256, bias_tok=256)) == 1    # no values
    assert process(rules(mask=256, mask_stride=3)) == 2
    verify = lambda ws=P, n=1 << 30, parent=P, tok=P: lib.logits_verify(P, 100, 4, 100, rules(), parent, parent, None, 1, tok,
                                                                        P, P, P, P, ws, n, None)
    assert verify(ws=None) == 1 and verify(n=0) == 3 and verify(parent=None) == 1 and verify(tok=None) == 1
    assert verify(ws=ctypes.c_void_p(260)) == 1
    assert lib.logits_verify_workspace_size(0, 100, 1) == 0
    assert lib.logits_verify_workspace_size(192, 151936, 24) >= 192 * 8


def test_workspace_sizes(w12):
    lib = w12.lib()
    assert lib.tree_attn_workspace_size(0, 1, 8, 8, 128) == 0
    assert lib.tree_attn_workspace_size(16, 1, 40, 8, 128) > 0


def test_slot_results_apart_from_what_is_read(w12):
    """Blocks read requests' numbers while others already write results."""
    names = ("len", "add", "table", "pool", "pos", "path", "off", "slot", "src", "new", "pos_out", "total", "status")
    size = dict(len=8, add=8, table=28, pool=32, pos=16, path=16, off=12, slot=64, src=32, new=8, pos_out=16, total=8, status=4)
    at = {n: 4096 * (i + 1) for i, n in enumerate(names)}

    def call(**kw):
        a = {n: ctypes.c_void_p(x) for n, x in dict(at, **kw).items()}
        return w12.lib().kv_slots(a["len"], a["add"], 0, 2, a["table"], 4, 3, a["pool"], 8, a["pos"], 16, a["path"], a["off"], 4,
                                  8, a["slot"], a["src"], a["new"], a["pos_out"], a["total"], a["status"], None)

    results = names[7:]
    for o in results:
        for n in names:
            if n != o:
                assert call(**{o: at[n]}) == 1, (o, n)
                assert call(**{o: at[n] + size[n] - 4}) == 1, (o, n)
                assert call(**{o: at[n] + 4 - size[o]}) == 1, (o, n)
                assert b"overlap" in w12.lib().w12_last_error() or (o, n) in (("new", "len"), ("pos_out", "pos"))


@pytest.mark.parametrize("scale", [2.4e38, 2.9e38, 3.4e38])
def test_scales_that_pass_the_largest_float_in_base_two(w12, scale):
    assert attn(w12, scale=scale) == 1
    assert b"scale" in w12.lib().w12_last_error()
