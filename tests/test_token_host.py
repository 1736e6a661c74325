"""Host-side checks of the packed-prompt and drafted-token calls: refusals come before any launch."""
import ctypes

import pytest
import torch

from block_sparse_attention_forecast_gb300 import build as _build

_build.build()

import block_sparse_attention_forecast_gb300.binding as sb  # noqa: E402

P = ctypes.c_void_p
FAKE, ODD = P(1 << 20), P((1 << 20) + 8)       # never dereferenced: the checks fail first
BIG = 1 << 40


def _shape(**kw):
    return sb.Shape(**{**dict(n_groups=2, heads_per_group=5, topk=8, max_ctx=4096, max_batch=2), **kw})


def _ref(s):
    return ctypes.byref(s.c())


def _layer(**kw):
    d = {**dict(k=1 << 20, v=1 << 20, ck=1 << 20, on_host=0), **kw}
    return ctypes.byref(sb.c_layer_kv(d["k"], d["v"], d["ck"], None, None, d["on_host"], 0))


def _prompt(shape=None, past=None, past_len=None, q=FAKE, qs=10 * 128, k=FAKE, v=FAKE, kvs=256, cu=FAKE, n=100, batch=1,
            out=FAKE, ws=FAKE, nws=BIG):
    return sb.lib.sparda_prompt_attn(_ref(shape or _shape()), past, past_len, q, qs, k, v, kvs, cu, n, batch, out, ws, nws, None)


def _tree(shape=None, layer=None, q=FAKE, qs=10 * 128, k=FAKE, v=FAKE, kvs=256, parent=FAKE, nodes=FAKE, n=8, idx=None,
          cnt=None, seq=FAKE, batch=1, out=FAKE, ws=FAKE, nws=BIG):
    return sb.lib.sparda_tree_attn(_ref(shape or _shape()), layer or _layer(), q, qs, k, v, kvs, parent, nodes, n, idx, cnt,
                                   seq, batch, out, ws, nws, None)


def _append(shape=None, layer=None, k=FAKE, v=FAKE, kvs=256, cu=FAKE, n=100, seq=FAKE, batch=1, new=None):
    return sb.lib.sparda_prompt_append(_ref(shape or _shape()), layer or _layer(), k, v, kvs, cu, n, seq, batch, new, None)


def _commit(shape=None, layer=None, k=FAKE, v=FAKE, kvs=256, n=8, path=FAKE, n_path=FAKE, seq=FAKE, batch=1, new=None):
    return sb.lib.sparda_tree_commit(_ref(shape or _shape()), layer or _layer(), k, v, kvs, n, path, n_path, seq, batch, new,
                                     None)


ALL = {"prompt": _prompt, "tree": _tree, "append": _append, "commit": _commit}


@pytest.mark.parametrize("name", ALL)
def test_shapes_and_batches(name):
    call = ALL[name]
    for bad in (dict(heads_per_group=17), dict(heads_per_group=0), dict(head_dim=64), dict(max_ctx=100), dict(block=128)):
        assert call(shape=_shape(**bad)) == sb.ERR_UNSUPPORTED_SHAPE, bad
    assert call(batch=0) == sb.ERR_INVALID_ARG
    assert call(batch=3) == sb.ERR_INVALID_ARG
    assert call(n=0) == sb.ERR_INVALID_ARG
    assert call(n=-1) == sb.ERR_INVALID_ARG
    assert call(n=(1 << 24) + 1 if name in ("prompt", "append") else 129) == sb.ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("name", ALL)
def test_rows(name):
    call = ALL[name]
    for t in ("k", "v") + (("q",) if name in ("prompt", "tree") else ()):
        assert call(**{t: None}) == sb.ERR_INVALID_ARG, t
        assert call(**{t: ODD}) == sb.ERR_MISALIGNED, t
    assert call(kvs=255) == sb.ERR_INVALID_ARG           # below a row's elements
    assert call(kvs=260) == sb.ERR_MISALIGNED            # rows off 16 bytes
    assert call(kvs=1 << 31) == sb.ERR_INVALID_ARG
    if name in ("prompt", "tree"):
        assert call(qs=10 * 128 - 8) == sb.ERR_INVALID_ARG
        assert call(qs=10 * 128 + 4) == sb.ERR_MISALIGNED
        assert call(out=None) == sb.ERR_INVALID_ARG and call(out=ODD) == sb.ERR_MISALIGNED
        assert call(ws=None) == sb.ERR_INVALID_ARG and call(ws=ODD) == sb.ERR_MISALIGNED
        kind = sb.WS_PROMPT if name == "prompt" else sb.WS_TREE
        need = sb.sparda_workspace_bytes(_shape(), 1, kind)
        assert need > 0 and call(nws=need - 1) == sb.ERR_WORKSPACE_TOO_SMALL


def test_layers_lengths_and_paths():
    for call in (_tree, _append, _commit):
        assert call(layer=_layer(k=None)) == sb.ERR_INVALID_ARG
        assert call(layer=_layer(v=(1 << 20) + 8)) == sb.ERR_MISALIGNED
        assert call(layer=_layer(on_host=1)) != sb.OK
    assert _prompt(past=_layer()) == sb.ERR_INVALID_ARG             # past without past_len, and the other way round
    assert _prompt(past_len=FAKE) == sb.ERR_INVALID_ARG
    assert _prompt(past=_layer(k=None), past_len=FAKE) == sb.ERR_INVALID_ARG
    assert _prompt(past=_layer(), past_len=P(2)) == sb.ERR_MISALIGNED
    assert _prompt(cu=None) == sb.ERR_INVALID_ARG and _prompt(cu=P(2)) == sb.ERR_MISALIGNED
    assert _append(cu=None) == sb.ERR_INVALID_ARG and _append(cu=P(2)) == sb.ERR_MISALIGNED
    assert _append(new=FAKE) == sb.ERR_INVALID_ARG                  # the lengths that are read
    assert _append(new=P(2)) == sb.ERR_MISALIGNED
    assert _commit(new=FAKE) == sb.ERR_INVALID_ARG
    assert _tree(seq=None) == sb.ERR_INVALID_ARG and _tree(seq=P(2)) == sb.ERR_MISALIGNED
    assert _tree(parent=P(2)) == sb.ERR_MISALIGNED and _tree(nodes=P(2)) == sb.ERR_MISALIGNED
    assert _tree(idx=FAKE) == sb.ERR_INVALID_ARG and _tree(cnt=FAKE) == sb.ERR_INVALID_ARG
    assert _tree(idx=P(2), cnt=FAKE) == sb.ERR_MISALIGNED
    for name in ("path", "n_path", "seq"):
        assert _commit(**{name: None}) == sb.ERR_INVALID_ARG, name
        assert _commit(**{name: P(2)}) == sb.ERR_MISALIGNED, name
    # a tensor map's last stride
    assert _prompt(n=1 << 24, qs=1 << 30) == sb.ERR_UNSUPPORTED_SHAPE


def test_lengths_that_no_counter_holds():
    # every second sequence may claim all tokens: 2^16 sequences, 2 groups, 41944 items of 25 tokens
    s = _shape(max_batch=1 << 16)
    assert _prompt(shape=s, n=1 << 20, batch=1 << 16) == sb.ERR_UNSUPPORTED_SHAPE


def test_workspaces():
    s = _shape()
    for kind in (sb.WS_PROMPT, sb.WS_TREE):
        n = sb.sparda_workspace_bytes(s, 2, kind)
        assert n == sb.sparda_workspace_bytes(s, 1, kind) > 2 * 152 * 256 * 130 * 4
        assert sb.sparda_workspace_bytes(s, 3, kind) == 0
        assert sb.sparda_workspace_bytes(_shape(heads_per_group=17), 1, kind) == 0


def test_binding_refuses_cpu_tensors():
    s = _shape()
    z = torch.zeros
    q, kv, cu = z(10, 10, 128, dtype=torch.bfloat16), z(10, 2, 128, dtype=torch.bfloat16), z(2, dtype=torch.int32)
    layer = sb.LayerKV(*(z(1, dtype=torch.bfloat16) for _ in range(3)))
    ws = z(16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        sb.sparda_prompt_attn(s, q, kv, kv, cu, 1, q, ws)
    with pytest.raises(ValueError):
        sb.sparda_prompt_append(s, layer, kv, kv, cu, None, 1)
    with pytest.raises(ValueError):
        sb.sparda_tree_attn(s, layer, q[None], kv[None], kv[None], None, cu, 1, q, ws)
    with pytest.raises(ValueError):
        sb.sparda_tree_commit(s, layer, kv[None], kv[None], cu, cu, cu, 1)
