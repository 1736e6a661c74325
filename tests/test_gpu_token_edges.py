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
NAN, INF = float("nan"), float("inf")


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


# ------------------------------------------------------------------------------- values that are not finite
def _formula(q, k, v, on, out, what):
    """out [n, D] against softmax(q k / sqrt(d)) v where keys may have one infinite channel: a score of -inf leaves its key
    out, and a row that has a score of +inf, or none but -inf, is NaN."""
    z = q @ k.T
    drop = torch.isinf(z)
    nan = (on & (z == INF)).any(dim=1) | ~(on & ~drop).any(dim=1)
    finite = torch.isfinite(k).all(dim=1, keepdim=True)
    want, bound = attend(q, torch.where(finite, k, torch.zeros_like(k)), v, on & ~drop)
    assert bool(torch.isnan(out[nan]).all()), what
    _check(out[~nan], want[~nan], bound[~nan], what)
    return int(nan.sum()), int((~nan).sum())


@pytest.mark.parametrize("lens,past,H", [([1, 1], None, 4), ([200, 31, 64], None, 16), ([400], [300], 2), ([5, 3], [6000, 6001], 3)], ids=str)
@pytest.mark.parametrize("every", [False, True])
def test_infinite_scores(lens, past, H, every):
    """Keys with an infinite channel, many in a row, and queries of either sign in it. every: all cached keys, and the new
    ones but every 50th."""
    G, B, rows = 1, len(lens), sum(lens)
    g = _gen(300 + rows)
    P = past or [0] * B
    shape = _shape(G, H, max(P + [64]), B)
    q, k, v = _projection((rows,), G, H, g)
    q[..., 0] = torch.where(torch.rand(q.shape[:-1], generator=g, device=DEV) < 0.1, 1.0, -1.0).to(torch.bfloat16)
    q[0, :, 0] = 1.0
    at = torch.arange(rows, device=DEV)
    k[(at % 50 != 49) if every else (at % 64 < 40), 0, 0] = INF
    layer, kw = None, {}
    if past:
        layer = _layer(shape, g, past)
        for b, n in enumerate(past):
            layer.k[b, :, : n if every else n // 2, 0] = INF
        kw = dict(past=layer, past_len=_i32(past))
    cu = [sum(lens[:i]) for i in range(B + 1)]
    out = torch.full((rows, G * H, D), 7.0, dtype=torch.bfloat16, device=DEV)
    sb.sparda_prompt_attn(shape, q, k, v, _i32(cu), B, out, sb.workspace(shape, B, sb.WS_PROMPT), **kw)
    seen = [0, 0]
    for b, n in enumerate(lens):
        part = slice(cu[b], cu[b + 1])
        kk, vv = k[part, 0].double(), v[part, 0].double()
        if past:
            kk, vv = torch.cat((layer.k[b, 0, : P[b]].double(), kk)), torch.cat((layer.v[b, 0, : P[b]].double(), vv))
        on = torch.ones((n, P[b] + n), dtype=torch.bool, device=DEV).tril(P[b])
        for h in range(H):
            for i, c in enumerate(_formula(q[part, h].double(), kk, vv, on, out[part, h], "sequence %d head %d" % (b, h))):
                seen[i] += c
    assert seen[0] > 0 and (seen[1] > 0 or rows < 10)
    assert sb.sparda_device_error() == 0


def test_tree_of_infinite_scores():
    G, H, N, ctx = 1, 4, 6, [0, 200]
    g = _gen(31)
    shape = _shape(G, H, 256, 2)
    layer = _layer(shape, g, ctx)
    layer.k[:, :, :200, 0] = INF
    q, k, v = _projection((2, N), G, H, g)
    q[..., 0] = -1.0
    k[:, [0, 1, 4], :, 0] = INF                                 # the root and two more: node 1 sees none but -inf
    parent = [-1, 0, 0, 1, 3, -1]
    out = torch.full((2, N, G * H, D), 7.0, dtype=torch.bfloat16, device=DEV)
    sb.sparda_tree_attn(shape, layer, q, k, v, _i32([parent] * 2), _i32(ctx), 2, out, sb.workspace(shape, 2, sb.WS_TREE))
    for b, S in enumerate(ctx):
        kk, vv = (torch.cat((c[b, 0, :S], x[b, :, 0])).double() for c, x in ((layer.k, k), (layer.v, v)))
        on = torch.cat((torch.ones((N, S), dtype=torch.bool), ancestors(parent, N)), dim=1).to(DEV)
        for h in range(H):
            nan, _ = _formula(q[b, :, h].double(), kk, vv, on, out[b, :, h], "sequence %d head %d" % (b, h))
            assert nan == 2
    assert sb.sparda_device_error() == 0


def test_attended_nan_and_infinite_values():
    """A NaN key reaches the rows that attend it, a NaN query its own row, a value its own channel."""
    G, H, n = 1, 3, 300
    g = _gen(32)
    shape = _shape(G, H, 64, 1)
    q, k, v = _projection((n,), G, H, g)
    ws = sb.workspace(shape, 1, sb.WS_PROMPT)
    want, out = (torch.empty((n, G * H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    call = lambda o: sb.sparda_prompt_attn(shape, q, k, v, _i32([0, n]), 1, o, ws)
    call(want)
    k[150, 0, 7], q[80, 1, 9] = NAN, NAN
    call(out)
    assert bool(torch.isnan(out[150:]).all()) and bool(torch.isnan(out[80, 1]).all())
    out[80, 1] = want[80, 1]
    assert torch.equal(out[:150], want[:150])
    k[150, 0, 7], q[80, 1, 9] = 0.0, 0.0
    call(want)
    v[20, 0, 3], v[90, 0, 4] = INF, NAN
    call(out)
    assert bool((out[20:, :, 3] == INF).all()) and bool(torch.isnan(out[90:, :, 4]).all())
    keep = [c for c in range(D) if c not in (3, 4)]
    assert torch.equal(out[..., keep], want[..., keep])
    assert sb.sparda_device_error() == 0


# ------------------------------------------------------------------------------- very large scores
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [2.0**14, 2.0**17, 2.0**38])
@pytest.mark.parametrize("n,past,H", [(70, 0, 16), (700, 0, 3), (6, 6000, 1)], ids=str)
def test_scores_far_beyond_the_exponents_of_probabilities(n, past, H, size, sign):
    """One channel is not zero, so that every score is exact: size^2 (1 + m/128) 2^e. Any two differ by far more than
    the exponents of float32: a row is the value of its largest key, exactly, or the mean of two values where two keys tie."""
    G = 1
    g = _gen(400 + n + past)
    shape = _shape(G, H, max(64, past), 1)
    q, k, v = _projection((n,), G, H, g)
    q.zero_()
    q[..., 5] = size
    # distinct keys in a random order (values of bf16); the last one of the whole once more
    m = torch.arange(past + n, device=DEV)
    m = m[torch.randperm(past + n, generator=g, device=DEV)]
    key = (size * (1 + (m % 128) / 128.0) * 2.0 ** (m // 128)).to(torch.bfloat16) * sign
    k.zero_()
    layer, kw = None, {}
    vv = v[:, 0]
    if past:
        layer = _layer(shape, g, [past])
        layer.k.zero_()
        layer.k[0, 0, :past, 5] = key[:past]
        kw = dict(past=layer, past_len=_i32([past]))
        vv = torch.cat((layer.v[0, 0, :past], vv))
    key[-1] = key[-2]
    k[:, 0, 5] = key[past:]
    out = torch.full((n, G * H, D), 7.0, dtype=torch.bfloat16, device=DEV)
    sb.sparda_prompt_attn(shape, q, k, v, _i32([0, n]), 1, out, sb.workspace(shape, 1, sb.WS_PROMPT), **kw)
    for i in range(n):
        seen = key[: past + i + 1].double()
        top = seen == seen.max()
        assert 1 <= int(top.sum()) <= 2
        want = vv[: past + i + 1][top].double().mean(dim=0)
        # the mean of two bf16 values: their sum in float32 rounds to 2^-24, then one rounding to bf16
        assert bool(((out[i].double() - want).abs() <= (2.0**-8 + 2.0**-20) * want.abs() * (int(top.sum()) - 1)).all()), i
    assert sb.sparda_device_error() == 0


@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("exponent", [31, 34, 36, 61])
@pytest.mark.parametrize("n,past,H", [(200, 0, 3), (4, 9000, 1)], ids=str)
def test_scores_one_step_of_float32_apart(n, past, H, exponent, order):
    """Exact scores 2^exponent (1.984375 + j 2^-23), j distinct: their products with log2(e) / sqrt(128) lie in the binade
    above, where neighbours round to one number. A step is 2^5 and more in log2 (exponent 31), so that a row is the value of
    its largest key to 2^-30."""
    G = 1
    g = _gen(500 + n)
    shape = _shape(G, H, max(64, past), 1)
    q, k, v = _projection((n,), G, H, g)
    total = past + n
    j = torch.arange(total, device=DEV)
    if order == "falling":
        j = j.flip(0)
    elif order == "mixed":
        j = j[torch.randperm(total, generator=g, device=DEV)]
    keys = torch.zeros((total, D), dtype=torch.bfloat16, device=DEV)
    keys[:, 0] = 1.984375 * 2.0 ** (exponent - 17)
    keys[:, 1] = (j % 256).float() * 2.0 ** (exponent - 40)
    keys[:, 2] = (j // 256).float() * 2.0 ** (exponent - 32)
    q.zero_()
    q[..., :3] = 2.0**17
    kw, vv = {}, v[:, 0]
    if past:
        layer = _layer(shape, g, [past])
        layer.k[0, 0, :past] = keys[:past]
        kw = dict(past=layer, past_len=_i32([past]))
        vv = torch.cat((layer.v[0, 0, :past], vv))
    k[:, 0] = keys[past:]
    score = (keys[:, :3].double() * 2.0**17).sum(dim=1)
    assert torch.equal(score.float().double(), score) and len(torch.unique(score)) == total
    out = torch.full((n, G * H, D), 7.0, dtype=torch.bfloat16, device=DEV)
    sb.sparda_prompt_attn(shape, q, k, v, _i32([0, n]), 1, out, sb.workspace(shape, 1, sb.WS_PROMPT), **kw)
    for i in range(n):
        want = vv[int(score[: past + i + 1].argmax())].double()
        # the other keys together: total * 2^-32 of their values, all below 8; then one rounding to bf16
        assert bool(((out[i].double() - want).abs() <= (2.0**-8) * want.abs() + total * 2.0**-32 * 16).all()), i
    assert sb.sparda_device_error() == 0
