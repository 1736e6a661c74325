"""Attention of new tokens and their store at their edges: references that move in a segment's last step, scores out of
the ordinary, values that are not finite, and rows that two sequences claim."""
import pytest
import torch

from tests.test_gpu_tokens import (_check, _clean_error_word, _copy, _gen, _i32, _layer, _projection, _randn, _shape,  # noqa: F401
                                   _store_check)
from tests.token_reference import D, ancestors, attend

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import block_sparse_attention_forecast_gb300.binding as sb

DEV = "cuda"


# ------------------------------------------------------------------------------- references
def _spread(q, k, gen, high=64.0):
    """Queries whose scores spread far beyond 2^7 (log2), and a few keys per 64 tokens that beat the others for some rows:
    rows and heads move their references at different keys, in either half of a key tile, the last one's too."""
    q[:] = q * high
    hot = torch.rand(k.shape[:-1], generator=gen, device=DEV) < 0.05
    k[:] = torch.where(hot[..., None], k * 4, k)


@pytest.mark.parametrize("lens", [[1], [2, 33, 64], [65, 100, 128], [129, 190, 192], [193, 256, 320]], ids=str)
@pytest.mark.parametrize("H", [1, 5, 16])
def test_references_that_move_in_the_last_key_tile(lens, H):
    """One key tile (the reference always moves there) and a few, the last of one block or two: against float64, and
    the same bits in every call."""
    G, B, rows = 2, len(lens), sum(lens)
    g = _gen(100 + H)
    shape = _shape(G, H, 64, B)
    q, k, v = _projection((rows,), G, H, g)
    _spread(q, k, g)
    cu, ws = _i32([sum(lens[:i]) for i in range(B + 1)]), sb.workspace(shape, B, sb.WS_PROMPT)
    out = torch.empty((rows, G * H, D), dtype=torch.bfloat16, device=DEV)
    sb.sparda_prompt_attn(shape, q, k, v, cu, B, out, ws)
    first = 0
    for b, n in enumerate(lens):
        at = slice(first, first + n)
        on = torch.ones((n, n), dtype=torch.bool, device=DEV).tril()
        for h in range(G * H):
            want, bound = attend(q[at, h].double(), k[at, h // H].double(), v[at, h // H].double(), on)
            _check(out[at, h], want, bound, "sequence %d head %d" % (b, h))
        first += n
    again = torch.empty_like(out)
    for _ in range(50):
        again.fill_(7.0)
        sb.sparda_prompt_attn(shape, q, k, v, cu, B, again, ws)
        assert torch.equal(again, out)
    assert sb.sparda_device_error() == 0


@pytest.mark.parametrize("ctx", [[0, 1, 64], [63, 65, 127], [1000, 5, 192]], ids=str)
@pytest.mark.parametrize("N,H", [(1, 16), (7, 3), (40, 16)])
def test_tree_references_that_move_in_the_last_key_tile(ctx, N, H):
    G, B = 2, len(ctx)
    g = _gen(200 + N)
    shape = _shape(G, H, max(ctx) + 64, B)
    layer = _layer(shape, g, ctx)
    q, k, v = _projection((B, N), G, H, g)
    _spread(q, k, g)
    parent = [-1] + [(i - 1) // 2 for i in range(1, N)]
    ws = sb.workspace(shape, B, sb.WS_TREE)
    out = torch.empty((B, N, G * H, D), dtype=torch.bfloat16, device=DEV)
    call = lambda o: sb.sparda_tree_attn(shape, layer, q, k, v, _i32([parent] * B), _i32(ctx), B, o, ws)
    call(out)
    for b, S in enumerate(ctx):
        on = torch.cat((torch.ones((N, S), dtype=torch.bool), ancestors(parent, N)), dim=1).to(DEV)
        for h in range(G * H):
            kk, vv = (torch.cat((c[b, h // H, :S], x[b, :, h // H])).double() for c, x in ((layer.k, k), (layer.v, v)))
            want, bound = attend(q[b, :, h].double(), kk, vv, on)
            _check(out[b, :, h], want, bound, "sequence %d head %d" % (b, h))
    again = torch.empty_like(out)
    for _ in range(50):
        again.fill_(7.0)
        call(again)
        assert torch.equal(again, out)
    assert sb.sparda_device_error() == 0


# ------------------------------------------------------------------------------- stores
@pytest.mark.parametrize("cu,start", [([0, 4096, 0, 4096], [0, 7, 45]),                      # one refused between two that hold all rows
                                      ([0, 2000, 100, 2000, 1, 1900, 1900], [64, 0, 1, 0, 31, 5]),
                                      ([0] + [1000, 3] * 40 + [1000], [b % 70 for b in range(81)])], ids=["two", "three", "forty-one"])
def test_rows_that_several_sequences_claim(cu, start):
    """Behind a sequence whose rows do not ascend, later ones may name rows again: every sequence that is not refused is
    stored whole, however many blocks of the cache that makes, and new_len says so."""
    G, B, n = 2, len(start), max(cu)
    g = _gen(B)
    shape = _shape(G, 3, max(start) + n, B)
    layer = _layer(shape, g, start)
    layer.ck.copy_(_randn(layer.ck.shape, g))
    _, k, v = _projection((n,), G, 3, g)
    before, new = _copy(layer), _i32([-5] * B)
    sb.sparda_prompt_append(shape, layer, k, v, _i32(cu), _i32(start), B, new_len=new)
    assert sb.sparda_device_error() == sb.DEV_BAD_SEQ_LEN
    good = [cu[b + 1] >= cu[b] for b in range(B)]
    assert sum(cu[b + 1] - cu[b] for b in range(B) if good[b]) > n
    for b in range(B):
        rows = slice(cu[b], cu[b + 1] if good[b] else cu[b])
        _store_check(layer, before, start[b], k[rows], v[rows], b)
        assert int(new[b]) == start[b] + rows.stop - rows.start
