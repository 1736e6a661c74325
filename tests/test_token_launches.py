"""Which kernels the packed-prompt and drafted-token calls launch, and what they do when a launch is refused: on the CPU,
against the stand-in for the CUDA runtime."""
import ctypes

import pytest

from tests.test_launch_errors import P, TOO_LARGE, compiled, sb


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    lib = compiled(str(tmp_path_factory.mktemp("tokens")), ["api.cu", "token_attn.cu", "token_append.cu"])
    for name in ("sparda_prompt_attn", "sparda_prompt_append", "sparda_tree_attn", "sparda_tree_commit"):
        getattr(lib, name).argtypes = getattr(sb.lib, name).argtypes
    return lib


def _names(lib):
    full = [lib.fake_launch(i).decode() for i in range(lib.fake_launches())]
    return [n[n.index("token_"):n.index("_kernel")] for n in full]


FAKE = P(1 << 20)


def _call(lib, kind, max_ctx=4096, batch=2, n=8):
    s = ctypes.byref(sb.Shape(n_groups=2, heads_per_group=16, topk=8, max_ctx=max_ctx, max_batch=batch).c())
    layer = ctypes.byref(sb.c_layer_kv(1 << 32, 1 << 33, 1 << 34, None, None, 0, 0))
    q, kv, room = 32 * 128, 2 * 128, 1 << 40
    if kind == "prompt":
        return lib.sparda_prompt_attn(s, None, None, FAKE, q, FAKE, FAKE, kv, FAKE, n, batch, FAKE, FAKE, room, None)
    if kind == "turn":
        return lib.sparda_prompt_attn(s, layer, FAKE, FAKE, q, FAKE, FAKE, kv, FAKE, n, batch, FAKE, FAKE, room, None)
    if kind == "tree":
        return lib.sparda_tree_attn(s, layer, FAKE, q, FAKE, FAKE, kv, FAKE, None, n, None, None, FAKE, batch, FAKE, FAKE, room, None)
    if kind == "append":
        return lib.sparda_prompt_append(s, layer, FAKE, FAKE, kv, FAKE, n, None, batch, None, None)
    return lib.sparda_tree_commit(s, layer, FAKE, FAKE, kv, n, FAKE, FAKE, FAKE, batch, None, None)


# (the kind, its sizes, its launches): what no call of the same arguments can cut has no join behind it, at most 8 blocks
CASES = [("prompt", dict(n=512), 1), ("prompt", dict(n=513), 2), ("prompt", dict(n=40, batch=20), 1), ("turn", dict(max_ctx=448, n=64), 1),
         ("turn", dict(max_ctx=512, n=64), 2), ("tree", dict(max_ctx=448, n=64), 1), ("tree", dict(max_ctx=448, n=65), 2), ("tree", {}, 2)]


@pytest.mark.parametrize("kind,sizes,n", CASES)
def test_an_attention_stops_at_a_refused_launch(lib, kind, sizes, n):
    """No join behind an attention that was refused, the call reports either refusal, and no error is left behind."""
    order = ["token_attn", "token_attn_join"][:n]
    for nth in range(n + 1):
        lib.fake_reset(nth, TOO_LARGE)
        assert _call(lib, kind, **sizes) == (sb.ERR_CUDA if nth < n else sb.OK), nth
        assert _names(lib) == order[:nth]
        assert lib.fake_last_error() == 0


@pytest.mark.parametrize("kind", ["append", "commit"])
def test_a_store_that_is_refused(lib, kind):
    lib.fake_reset(0, TOO_LARGE)
    assert _call(lib, kind) == sb.ERR_CUDA and _names(lib) == [] and lib.fake_last_error() == 0
    lib.fake_reset(-1, 0)
    assert _call(lib, kind) == sb.OK and _names(lib) == ["token_append"]
