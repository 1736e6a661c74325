"""Attention of packed prompts and of trees of drafted tokens, and their store into the cache, against float64."""
import pytest
import torch

from tests.token_reference import BLOCK, D, ancestors, attend, window_mean

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import block_sparse_attention_forecast_gb300.binding as sb

DEV = "cuda"
NAN = float("nan")


@pytest.fixture(autouse=True)
def _clean_error_word():
    sb.sparda_device_error()
    yield


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _shape(G, H, ctx, B, topk=8):
    return sb.Shape(n_groups=G, heads_per_group=H, topk=topk, max_ctx=(max(ctx, 1) + 63) // 64 * 64, max_batch=B)


def _layer(shape, g, lens, extra=0):
    """A resident layer whose rows past lens hold NaN."""
    layer = sb.LayerKV.empty(shape)
    for t in (layer.k, layer.v):
        t.copy_(_randn(t.shape, g))
        for b, n in enumerate(lens):
            t[b, :, n:] = NAN
    return layer


def _projection(lead, G, H, g, strided=True):
    """(q, k, v) of new tokens, slices of one projection or dense."""
    x = _randn((*lead, G * H + 2 * G, D), g)
    parts = x[..., : G * H, :], x[..., G * H : G * H + G, :], x[..., G * H + G :, :]
    return parts if strided else tuple(p.contiguous() for p in parts)


def _check(out, want, bound, what):
    err = (out.double() - want).abs()
    assert bool(torch.isfinite(out).all()), what
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert worst <= 1.0, "%s: %.3f of the bound" % (what, worst)


def _prompt_case(lens, past, G, H, seed, strided=True, ws=None, out=None, behind=3, scale=1.0, stream=None):
    g = _gen(seed)
    B = len(lens)
    shape = _shape(G, H, max(past) if past else 64, B)
    rows = sum(lens) + behind
    q, k, v = _projection((rows,), G, H, g, strided)
    q[:] = q * scale
    q[sum(lens):], k[sum(lens):], v[sum(lens):] = NAN, NAN, NAN
    cu = _i32([sum(lens[:i]) for i in range(B + 1)])
    ws = sb.workspace(shape, B, sb.WS_PROMPT) if ws is None else ws
    out = torch.full((rows, G * H, D), 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    kw = {}
    if past:
        layer = _layer(shape, g, past)
        kw = dict(past=layer, past_len=_i32(past))
    sb.sparda_prompt_attn(shape, q, k, v, cu, B, out, ws, **kw)
    torch.cuda.synchronize()
    assert sb.sparda_device_error() == 0
    assert bool((out[sum(lens):] == 7.0).all())
    first = 0
    for b, n in enumerate(lens):
        S = past[b] if past else 0
        on = torch.ones((n, S + n), dtype=torch.bool, device=DEV).tril(S)
        for gr in range(G):
            kk, vv = k[first : first + n, gr].double(), v[first : first + n, gr].double()
            if S:
                kk, vv = torch.cat((layer.k[b, gr, :S].double(), kk)), torch.cat((layer.v[b, gr, :S].double(), vv))
            for h in range(gr * H, gr * H + H):
                want, bound = attend(q[first : first + n, h].double(), kk, vv, on)
                _check(out[first : first + n, h], want, bound, "sequence %d head %d" % (b, h))
        first += n
    return ws


# ------------------------------------------------------------------------------- prompts
@pytest.mark.parametrize("H", [1, 2, 3, 5, 8, 11, 16])
@pytest.mark.parametrize("lens", [[1], [63, 0, 65], [64, 130, 1, 7], [300]], ids=str)
def test_prompt_heads_and_lengths(H, lens):
    _prompt_case(lens, None, 2, H, seed=17 * H + len(lens))


@pytest.mark.parametrize("past", [[0, 64, 1], [63, 200, 65], [128, 0, 1000]], ids=str)
@pytest.mark.parametrize("G,H", [(1, 16), (3, 4), (2, 1)])
def test_prompt_over_a_past(G, H, past):
    _prompt_case([70, 1, 129], past, G, H, seed=G + H, strided=(G != 3))


def test_prompt_whole_items_from_the_queue():
    # more items than are cut: 8 sequences x 4 groups x 32 items, shorter and longer ones
    _prompt_case([500, 333, 512, 17, 499, 256, 430, 388], None, 4, 16, seed=3)


@pytest.mark.parametrize("lens,G,H", [([3, 9, 14] * 19, 8, 16), ([2, 1] * 40, 8, 1), ([600] * 5, 8, 16)], ids=str)
def test_prompt_queue_is_left_at_zero(lens, G, H):
    # more items than run at once: without a call for joining and one query tile or two, and with it
    ws = None
    for seed in (5, 6):
        ws = _prompt_case(lens, None, G, H, seed=seed, ws=ws)
        assert not ws[:256].any()


@pytest.mark.parametrize("lens,past,G,H", [([100] + [0, 1] * 20, [700] + [65, 128] * 20, 2, 16), ([1] * 9 + [700], None, 3, 1),
                                           ([2000] + [5] * 300, None, 1, 16), ([1] * 33, [4096, 1, 0] * 11, 4, 5)],
                         ids=["turn", "heads of one", "long", "single tokens"])
def test_prompt_short_sequences_on_average(lens, past, G, H):
    # one query tile at a time, also for a sequence that is longer than the others
    _prompt_case(lens, past, G, H, seed=len(lens))


def test_prompt_few_long_items_are_cut():
    # one group and head: 8 items of up to 16 key tiles and a past of 90 more, shared by all SMs
    _prompt_case([2000], [11500], 1, 1, seed=4)
    _prompt_case([5], [12001], 1, 3, seed=5)           # items of many key tiles


def test_prompt_items_of_two_rounds_are_cut():
    # 160 items of 1 to 40 key tiles: ranges of several items, some of which end before an item's first key tile
    _prompt_case([5000], None, 8, 1, seed=6)


def test_prompt_scores_that_grow():
    # keys whose scores rise by more than 2^8 from tile to tile: the reference moves again and again
    G, H, n = 1, 4, 700
    g = _gen(8)
    shape = _shape(G, H, 64, 1)
    q, k, v = _projection((n,), G, H, g, strided=False)
    q[:] = 1.0
    k[:] = (torch.arange(n, device=DEV, dtype=torch.float32)[:, None, None] / 8).to(torch.bfloat16)
    out = torch.empty((n, G * H, D), dtype=torch.bfloat16, device=DEV)
    sb.sparda_prompt_attn(shape, q, k, v, _i32([0, n]), 1, out, sb.workspace(shape, 1, sb.WS_PROMPT))
    on = torch.ones((n, n), dtype=torch.bool, device=DEV).tril()
    for h in range(H):
        want, bound = attend(q[:, h].double(), k[:, 0].double(), v[:, 0].double(), on)
        _check(out[:, h], want, bound, "head %d" % h)
    # falling ones, and scores of one large value each
    k[:] = torch.flip(k, (0,))
    sb.sparda_prompt_attn(shape, q, k, v, _i32([0, n]), 1, out, sb.workspace(shape, 1, sb.WS_PROMPT))
    for h in range(H):
        want, bound = attend(q[:, h].double(), k[:, 0].double(), v[:, 0].double(), on)
        _check(out[:, h], want, bound, "falling, head %d" % h)


def test_prompt_sequences_do_not_reach_each_other():
    G, H, lens = 2, 16, [100, 90, 50]
    g = _gen(9)
    shape = _shape(G, H, 64, 3)
    q, k, v = _projection((240,), G, H, g)
    cu = _i32([0, 100, 190, 240])
    ws = sb.workspace(shape, 3, sb.WS_PROMPT)
    want, out = (torch.empty((240, G * H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sb.sparda_prompt_attn(shape, q, k, v, cu, 3, want, ws)
    q[100:190], k[100:190], v[100:190] = float("inf"), NAN, float("-inf")
    sb.sparda_prompt_attn(shape, q, k, v, cu, 3, out, ws)
    assert torch.equal(out[:100], want[:100]) and torch.equal(out[190:], want[190:])


def test_prompt_bad_lengths():
    G, H, B = 2, 4, 4
    g = _gen(10)
    shape = _shape(G, H, 128, B)
    q, k, v = _projection((200,), G, H, g)
    layer = _layer(shape, g, [128] * B)
    ws = sb.workspace(shape, B, sb.WS_PROMPT)
    out = torch.full((200, G * H, D), 7.0, dtype=torch.bfloat16, device=DEV)
    # sequence 1 ends behind the rows, sequence 2 begins behind its end; 0 and 3 have a past out of range
    sb.sparda_prompt_attn(shape, q, k, v, _i32([0, 50, 201, 100, 150]), B, out, ws, past=layer, past_len=_i32([-1, 0, 0, 129]))
    assert sb.sparda_device_error() == sb.DEV_BAD_SEQ_LEN
    assert bool((out == 7.0).all())
    sb.sparda_prompt_attn(shape, q, k, v, _i32([0, 50, 50, 40, 90]), B, out, ws, past=layer, past_len=_i32([0, 0, 0, 128]))
    assert sb.sparda_device_error() == sb.DEV_BAD_SEQ_LEN                      # (sequence 2 alone)
    assert bool((out[:90] != 7.0).any()) and bool((out[90:] == 7.0).all())


# ------------------------------------------------------------------------------- trees
def _tree_case(ctx, nodes, N, G, H, kind, seed, topk=0, strided=True, ws=None):
    g = _gen(seed)
    B = len(ctx)
    shape = _shape(G, H, max(ctx) + 64, B, topk=max(1, topk))
    layer = _layer(shape, g, ctx)
    q, k, v = _projection((B, N), G, H, g, strided)
    for b, n in enumerate(nodes):
        q[b, n:], k[b, n:], v[b, n:] = NAN, NAN, NAN
    rnd = torch.Generator()
    rnd.manual_seed(seed)
    parent = None
    if kind == "random":
        parent = [[-1 if i == 0 else int(torch.randint(max(-1, i - 9), i, (1,), generator=rnd)) for i in range(N)] for _ in ctx]
    elif kind == "roots":
        parent = [[-1] * N for _ in ctx]
    elif kind == "line":
        parent = [[i - 1 for i in range(N)] for _ in ctx]
    kw = {}
    if topk:
        nb = shape.max_ctx // BLOCK
        idx = torch.full((B, G, topk + 2), -1, dtype=torch.int32)
        cnt = torch.zeros((B, G), dtype=torch.int32)
        for b, S in enumerate(ctx):
            for gr in range(G):
                last = S // BLOCK
                pick = sorted({0, last} | set(torch.randperm(last + 1, generator=rnd)[:topk].tolist()))[: topk + 2]
                if gr == 0 and len(pick) > 2:
                    pick[1] = pick[2]                       # a block named twice counts twice
                idx[b, gr, : len(pick)] = torch.tensor(pick, dtype=torch.int32)
                cnt[b, gr] = len(pick)
        cnt[-1, -1] = 0                                     # nothing of the cache
        kw = dict(idx=idx.to(DEV), cnt=cnt.to(DEV))
        assert nb > 0
    out = torch.full((B, N, G * H, D), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = sb.workspace(shape, B, sb.WS_TREE) if ws is None else ws
    sb.sparda_tree_attn(shape, layer, q, k, v, None if parent is None else _i32(parent), _i32(ctx), B, out, ws,
                        n_nodes=None if all(n == N for n in nodes) else _i32(nodes), **kw)
    torch.cuda.synchronize()
    assert sb.sparda_device_error() == 0
    for b, (S, n) in enumerate(zip(ctx, nodes)):
        assert bool((out[b, n:] == 7.0).all())
        line = ancestors(None if parent is None else parent[b], n).to(DEV)
        for gr in range(G):
            if topk:
                at = [j * BLOCK + e for j in kw["idx"][b, gr, : int(kw["cnt"][b, gr])].tolist() for e in range(BLOCK) if j * BLOCK + e < S]
                at = torch.tensor(at, dtype=torch.long, device=DEV)
            else:
                at = torch.arange(S, device=DEV)
            kk = torch.cat((layer.k[b, gr, at].double(), k[b, :n, gr].double()))
            vv = torch.cat((layer.v[b, gr, at].double(), v[b, :n, gr].double()))
            on = torch.cat((torch.ones((n, len(at)), dtype=torch.bool, device=DEV), line), dim=1)
            for h in range(gr * H, gr * H + H):
                want, bound = attend(q[b, :n, h].double(), kk, vv, on)
                _check(out[b, :n, h], want, bound, "sequence %d head %d" % (b, h))
    return ws


@pytest.mark.parametrize("kind", ["random", "chain", "roots", "line"])
@pytest.mark.parametrize("N,H", [(1, 16), (2, 1), (8, 16), (9, 16), (17, 5), (64, 4), (65, 2), (128, 16)])
def test_tree_shapes(kind, N, H):
    _tree_case([0, 1, 64, 130], [N, max(0, N - 1), N, N // 2], N, 2, H, kind, seed=N + H)


@pytest.mark.parametrize("ctx", [[63, 65], [1000], [5000, 128, 0], [20000]], ids=str)
@pytest.mark.parametrize("N,G,H", [(1, 2, 16), (5, 3, 7), (40, 1, 16)])
def test_tree_contexts(ctx, N, G, H):
    _tree_case(ctx, [N] * len(ctx), N, G, H, "random", seed=ctx[0] + N, strided=(G != 3))


@pytest.mark.parametrize("topk", [1, 7, 62])
@pytest.mark.parametrize("N,H", [(1, 16), (6, 5), (33, 16)])
def test_tree_over_selected_blocks(topk, N, H):
    _tree_case([64 * 70, 5000, 63, 64], [N, N, max(1, N - 1), N], N, 2, H, "random", seed=topk + N, topk=topk)


def test_tree_many_sequences():
    # more entries than lanes, items from the queue
    g = torch.Generator()
    g.manual_seed(5)
    ctx = torch.randint(0, 400, (70,), generator=g).tolist()
    nodes = torch.randint(0, 21, (70,), generator=g).tolist()
    _tree_case(ctx, nodes, 20, 3, 16, "random", seed=6)


def test_tree_bad_inputs():
    G, H, N, B = 2, 4, 6, 3
    g = _gen(12)
    shape = _shape(G, H, 256, B, topk=2)
    layer = _layer(shape, g, [100, 200, 256])
    q, k, v = _projection((B, N), G, H, g)
    ws = sb.workspace(shape, B, sb.WS_TREE)
    good = [[-1, 0, 1, 0, 3, -1]] * B
    want = torch.full((B, N, G * H, D), 7.0, dtype=torch.bfloat16, device=DEV)
    sb.sparda_tree_attn(shape, layer, q, k, v, _i32(good), _i32([100, 200, 256]), B, want, ws)
    assert sb.sparda_device_error() == 0
    # parents that are no lower node count as -1
    out = torch.full_like(want, 7.0)
    sb.sparda_tree_attn(shape, layer, q, k, v, _i32([[0, 0, 1, 0, 3, 99], [-7, 0, 1, 0, 3, 5], [1 << 30, 0, 1, 0, 3, 6]]),
                        _i32([100, 200, 256]), B, out, ws)
    assert sb.sparda_device_error() == sb.DEV_BAD_INDEX
    assert torch.equal(out, want)
    # lengths out of range write nothing
    out.fill_(7.0)
    sb.sparda_tree_attn(shape, layer, q, k, v, _i32(good), _i32([-1, 200, 257]), B, out, ws)
    assert sb.sparda_device_error() == sb.DEV_BAD_SEQ_LEN
    assert bool((out[0] == 7.0).all()) and bool((out[2] == 7.0).all()) and torch.equal(out[1], want[1])
    out.fill_(7.0)
    sb.sparda_tree_attn(shape, layer, q, k, v, _i32(good), _i32([100, 200, 256]), B, out, ws, n_nodes=_i32([-1, 6, 7]))
    assert sb.sparda_device_error() == sb.DEV_BAD_SEQ_LEN
    assert bool((out[0] == 7.0).all()) and bool((out[2] == 7.0).all()) and torch.equal(out[1], want[1])
    # blocks outside the sequence are skipped: block 2 of 100 tokens, and a fourth that no sequence has
    idx = torch.tensor([0, 1, 2, 1000000], dtype=torch.int32, device=DEV).expand(B, G, 4).contiguous()
    for n in (3, 4):
        cnt = torch.full((B, G), n, dtype=torch.int32, device=DEV)
        sb.sparda_tree_attn(shape, layer, q, k, v, _i32(good), _i32([100, 200, 256]), B, out, ws, idx=idx, cnt=cnt)
        assert sb.sparda_device_error() == sb.DEV_BAD_INDEX
        for b, S in enumerate((100, 192, 192)):
            on = torch.cat((torch.ones((N, S), dtype=torch.bool, device=DEV), ancestors(good[b], N).to(DEV)), dim=1)
            for h in range(G * H):
                kk = torch.cat((layer.k[b, h // H, :S], k[b, :, h // H])).double()
                vv = torch.cat((layer.v[b, h // H, :S], v[b, :, h // H])).double()
                ref, bound = attend(q[b, :, h].double(), kk, vv, on)
                _check(out[b, :, h], ref, bound, "sequence %d head %d" % (b, h))


def test_one_node_is_the_decode_step():
    """A single node over selected blocks gives the decode attention's result on the stored token, within the two
    kernels' bounds."""
    G, H, B, T = 2, 16, 4, 3000
    g = _gen(13)
    shape = sb.Shape(n_groups=G, heads_per_group=H, topk=10, max_ctx=4096, max_batch=B)
    layer = _layer(shape, g, [T - 1] * B)
    layer.k[:, :, T - 1 :], layer.v[:, :, T - 1 :] = 0.0, 0.0
    q, k, v = _projection((B, 1), G, H, g, strided=False)
    idx = torch.full((B, G, 12), -1, dtype=torch.int32, device=DEV)
    idx[..., :5] = _i32([0, 3, 7, 20, (T - 1) // 64])
    cnt = torch.full((B, G), 5, dtype=torch.int32, device=DEV)
    out = torch.empty((B, 1, G * H, D), dtype=torch.bfloat16, device=DEV)
    sb.sparda_tree_attn(shape, layer, q, k, v, None, _i32([T - 1] * B), B, out, sb.workspace(shape, B, sb.WS_TREE), idx=idx, cnt=cnt)
    sb.sparda_append_kv(shape, layer, k.view(B, G, D), v.view(B, G, D), _i32([T] * B), B)
    ref = torch.empty((B, G * H, D), dtype=torch.bfloat16, device=DEV)
    sb.sparda_sparse_decode_attn(shape, layer, q.view(B, G * H, D), idx, cnt, _i32([T] * B), B, ref, sb.workspace(shape, B, sb.WS_ATTN))
    at = torch.cat([torch.arange(j * 64, min(T, j * 64 + 64), device=DEV) for j in (0, 3, 7, 20, (T - 1) // 64)])
    for b in range(B):
        for h in range(G * H):
            kk, vv = layer.k[b, h // H, at].double(), layer.v[b, h // H, at].double()
            on = torch.ones((1, len(at)), dtype=torch.bool, device=DEV)
            want, bound = attend(q[b, :, h].double(), kk, vv, on)
            _check(out[b, :, h], want, bound, "sequence %d head %d" % (b, h))
            _check(ref[b : b + 1, h], want, bound, "decode, sequence %d head %d" % (b, h))


# ------------------------------------------------------------------------------- stores
def _store_check(layer, before, S, keys, values, b):
    """Sequence b of `layer` holds `before` with keys / values [n, G, D] behind its first S tokens."""
    n = keys.shape[0]
    k, v, ck = (t[b].clone() for t in (before.k, before.v, before.ck))
    k[:, S : S + n], v[:, S : S + n] = keys.transpose(0, 1), values.transpose(0, 1)
    for end in range(32, S + n + 1, 16):
        if end > S:
            ck[:, (end - 32) // 16] = window_mean(k[:, end - 32 : end].transpose(0, 1))
    eq = lambda x, y: torch.equal(x.view(torch.int16), y.view(torch.int16))     # NaN bits included
    assert eq(layer.k[b], k) and eq(layer.v[b], v)
    assert eq(layer.ck[b], ck)


def _copy(layer):
    return sb.LayerKV(layer.k.clone(), layer.v.clone(), layer.ck.clone())


@pytest.mark.parametrize("lens,start", [([1], [0]), ([33, 0, 31], [0, 5, 1]), ([130, 64, 1], [63, 64, 15]),
                                        ([500, 17, 100], [1000, 31, 47])], ids=str)
@pytest.mark.parametrize("G,strided", [(1, True), (3, False)])
def test_prompt_append(lens, start, G, strided):
    g = _gen(len(lens) + G)
    B = len(lens) + 1                                  # one sequence more than the call's: untouched
    shape = _shape(G, 3, 1600, B)
    layer = _layer(shape, g, start + [0])
    layer.ck.copy_(_randn(layer.ck.shape, g))
    _, k, v = _projection((sum(lens) + 2,), G, 3, g, strided)
    before = _copy(layer)
    new = _i32([-5] * (B - 1))
    empty = all(s == 0 for s in start)
    sb.sparda_prompt_append(shape, layer, k, v, _i32([sum(lens[:i]) for i in range(B)]), None if empty else _i32(start), B - 1,
                            new_len=new)
    assert sb.sparda_device_error() == 0
    assert new.tolist() == [s + n for s, n in zip(start, lens)]
    first = 0
    for b, n in enumerate(lens):
        _store_check(layer, before, start[b], k[first : first + n], v[first : first + n], b)
        first += n
    _store_check(layer, before, 0, k[:0], v[:0], B - 1)


def test_append_of_extreme_keys():
    """Compressed keys of windows whose keys differ by many powers of two, cancel or are not finite."""
    g = _gen(21)
    shape = _shape(2, 1, 256, 1)
    layer = _layer(shape, g, [0])
    _, k, v = _projection((200,), 2, 1, g, strided=False)
    k[:64] = k[:64] * (2.0 ** torch.randint(-30, 9, (64, 2, D), generator=g, device=DEV)).to(torch.bfloat16)
    k[64:96] = torch.where(torch.arange(32, device=DEV)[:, None, None] % 2 == 0, 3.0, -3.0).to(torch.bfloat16)
    before = _copy(layer)
    sb.sparda_prompt_append(shape, layer, k, v, _i32([0, 200]), None, 1)
    _store_check(layer, before, 0, k, v, 0)
    k[150, 0, 5], k[151, 1, 7] = float("inf"), NAN
    sb.sparda_prompt_append(shape, layer, k, v, _i32([0, 200]), None, 1)
    ck = layer.ck[0].float()
    assert float(ck[0, 8, 5]) == float("inf") and bool(torch.isnan(ck[1, 8, 7]))       # tokens 128 .. 159
    assert bool(torch.isfinite(ck[:, :7]).all())


@pytest.mark.parametrize("N", [1, 7, 64, 128])
def test_tree_commit_is_many_appends(N):
    G, B = 2, 4
    g = _gen(N)
    start = [0, 31, 64, 777]
    shape = sb.Shape(n_groups=G, heads_per_group=16, topk=8, max_ctx=1024, max_batch=B)
    layer = _layer(shape, g, start)
    layer.ck.copy_(_randn(layer.ck.shape, g))
    _, k, v = _projection((B, N), G, 16, g)
    rnd = torch.Generator()
    rnd.manual_seed(N)
    paths = [sorted(torch.randperm(N, generator=rnd)[: [N, 0, (N + 1) // 2, max(1, N // 3)][b]].tolist()) for b in range(B)]
    one = _copy(layer)
    before = _copy(layer)
    new = _i32([0] * B)
    sb.sparda_tree_commit(shape, layer, k, v, _i32([p + [-1] * (N - len(p)) for p in paths]), _i32([len(p) for p in paths]),
                          _i32(start), B, new_len=new)
    assert sb.sparda_device_error() == 0
    assert new.tolist() == [s + len(p) for s, p in zip(start, paths)]
    for b in range(B):
        at = torch.tensor(paths[b], dtype=torch.long, device=DEV)
        _store_check(layer, before, start[b], k[b, at], v[b, at], b)
        # token by token (the caches of one sequence as a batch of one)
        sub = sb.LayerKV(one.k[b : b + 1], one.v[b : b + 1], one.ck[b : b + 1])
        for i, node in enumerate(paths[b]):
            sb.sparda_append_kv(shape, sub, k[b, node].contiguous(), v[b, node].contiguous(), _i32([start[b] + i + 1]), 1)
    for x, y in ((layer.k, one.k), (layer.v, one.v), (layer.ck, one.ck)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_store_bad_inputs_leave_the_cache():
    G, B, N = 2, 4, 8
    g = _gen(30)
    shape = sb.Shape(n_groups=G, heads_per_group=16, topk=8, max_ctx=256, max_batch=B)
    layer = _layer(shape, g, [100] * B)
    layer.ck.copy_(_randn(layer.ck.shape, g))
    before = _copy(layer)
    _, k, v = _projection((B, N), G, 16, g)
    path = [[0, 1, 2, 3, 4, 5, 6, 7]] * B
    new = _i32([0] * B)
    same = lambda b: all(torch.equal(x[b].view(torch.int16), y[b].view(torch.int16))
                         for x, y in ((layer.k, before.k), (layer.v, before.v), (layer.ck, before.ck)))
    # no room, a negative length, a path longer than the tree, and a good one
    sb.sparda_tree_commit(shape, layer, k, v, _i32(path), _i32([8, 8, 9, 8]), _i32([249, -1, 100, 100]), B, new_len=new)
    assert sb.sparda_device_error() == sb.DEV_BAD_SEQ_LEN
    assert same(0) and same(1) and same(2) and not same(3)
    assert new.tolist() == [249, -1, 100, 108]
    layer = _copy(before)
    bad = [list(p) for p in path]
    bad[0][3], bad[2][7] = 8, -1
    sb.sparda_tree_commit(shape, layer, k, v, _i32(bad), _i32([8, 8, 8, 3]), _i32([100] * B), B, new_len=new)
    assert sb.sparda_device_error() == sb.DEV_BAD_INDEX
    assert same(0) and not same(1) and same(2) and not same(3)
    assert new.tolist() == [100, 108, 100, 103]
    layer = _copy(before)
    kk, vv = k.reshape(B * N, G, D), v.reshape(B * N, G, D)
    sb.sparda_prompt_append(shape, layer, kk, vv, _i32([0, 8, 40, 30, 33]), _i32([250, 100, 100, 256]), B, new_len=new)
    assert sb.sparda_device_error() == sb.DEV_BAD_SEQ_LEN
    assert all(same(b) for b in range(B))


# ------------------------------------------------------------------------------- as a user runs them
@pytest.mark.parametrize("H", [16, 5])
def test_a_conversation(H):
    """Prompts attended and stored, a second turn on top, drafts verified and committed, and the next draft: every
    attention against float64 over the tokens so far, the caches against a cache filled at once."""
    G, B, N = 2, 3, 12
    g = _gen(40 + H)
    shape = sb.Shape(n_groups=G, heads_per_group=H, topk=8, max_ctx=1024, max_batch=B)
    layer = sb.LayerKV.empty(shape)
    for t in (layer.k, layer.v):
        t.fill_(NAN)
    ws_p, ws_t = sb.workspace(shape, B, sb.WS_PROMPT), sb.workspace(shape, B, sb.WS_TREE)
    keys, values = ([torch.zeros((0, G, D), dtype=torch.bfloat16, device=DEV) for _ in range(B)] for _ in range(2))
    seq, spare = _i32([0] * B), _i32([0] * B)

    def check(out, q, k, v, b, on_new):
        n = q.shape[0]
        S = keys[b].shape[0]
        on = torch.cat((torch.ones((n, S), dtype=torch.bool, device=DEV), on_new.to(DEV)), dim=1)
        for h in range(G * H):
            kk = torch.cat((keys[b][:, h // H], k[:, h // H])).double()
            vv = torch.cat((values[b][:, h // H], v[:, h // H])).double()
            want, bound = attend(q[:, h].double(), kk, vv, on)
            _check(out[:, h], want, bound, "sequence %d head %d" % (b, h))

    for lens in ([200, 33, 64], [5, 130, 0]):
        q, k, v = _projection((sum(lens),), G, H, g)
        cu = _i32([0, lens[0], lens[0] + lens[1], sum(lens)])
        out = torch.empty((sum(lens), G * H, D), dtype=torch.bfloat16, device=DEV)
        sb.sparda_prompt_attn(shape, q, k, v, cu, B, out, ws_p, past=layer, past_len=seq)
        sb.sparda_prompt_append(shape, layer, k, v, cu, seq, B, new_len=spare)
        seq, spare = spare, seq
        first = 0
        for b, n in enumerate(lens):
            part = slice(first, first + n)
            check(out[part], q[part], k[part], v[part], b, torch.ones((n, n), dtype=torch.bool).tril())
            keys[b], values[b] = torch.cat((keys[b], k[part])), torch.cat((values[b], v[part]))
            first += n
    rnd = torch.Generator()
    rnd.manual_seed(H)
    for step in range(3):
        q, k, v = _projection((B, N), G, H, g)
        parent = [[-1] + [int(torch.randint(0, i, (1,), generator=rnd)) for i in range(1, N)] for _ in range(B)]
        out = torch.empty((B, N, G * H, D), dtype=torch.bfloat16, device=DEV)
        sb.sparda_tree_attn(shape, layer, q, k, v, _i32(parent), seq, B, out, ws_t)
        paths = []
        for b in range(B):
            check(out[b], q[b], k[b], v[b], b, ancestors(parent[b], N))
            at, path = N - 1 - b, []
            while at >= 0:
                path.append(at)
                at = parent[b][at]
            paths.append(path[::-1])
        sb.sparda_tree_commit(shape, layer, k, v, _i32([p + [0] * (N - len(p)) for p in paths]), _i32([len(p) for p in paths]),
                              seq, B, new_len=spare)
        seq, spare = spare, seq
        for b in range(B):
            at = torch.tensor(paths[b], device=DEV)
            keys[b], values[b] = torch.cat((keys[b], k[b, at])), torch.cat((values[b], v[b, at]))
    assert sb.sparda_device_error() == 0
    assert seq.tolist() == [x.shape[0] for x in keys]
    full = sb.LayerKV(layer.k.clone(), layer.v.clone(), torch.zeros_like(layer.ck))
    sb.sparda_compress_keys(sb.Shape(n_groups=G, heads_per_group=16, topk=8, max_ctx=1024, max_batch=B), full, seq, B)
    for b in range(B):
        n = keys[b].shape[0]
        assert torch.equal(layer.k[b, :, :n], keys[b].transpose(0, 1)) and bool(torch.isnan(layer.k[b, :, n:]).all())
        assert torch.equal(layer.v[b, :, :n], values[b].transpose(0, 1))
        w = sb.num_windows(n)
        assert torch.equal(layer.ck[b, :, :w], full.ck[b, :, :w])


def test_store_prompt_and_selection_back_to_back():
    # a selection reads compressed keys ahead of its wait: what the store before a one-launch prompt wrote is there by then
    G, H, B, T = 2, 16, 2, 4000
    g = _gen(77)
    shape = sb.Shape(n_groups=G, heads_per_group=H, topk=16, max_ctx=4096, max_batch=B)
    layer = sb.LayerKV.empty(shape)
    q, k, v = _projection((2 * T,), G, H, g)
    forecasts = _randn((B, G, D), g)
    cu, cu_q, seq = _i32([0, T, 2 * T]), _i32([0, 40, 90]), _i32([T, T])
    out = torch.empty((90, G * H, D), dtype=torch.bfloat16, device=DEV)
    ws, ws_s = sb.workspace(shape, B, sb.WS_PROMPT), sb.workspace(shape, B, sb.WS_SELECT)

    def run(idx, cnt, between):
        sb.sparda_prompt_append(shape, layer, k, v, cu, None, B)
        between()
        sb.sparda_prompt_attn(shape, q[:90], k[:90], v[:90], cu_q, B, out, ws)
        between()
        sb.sparda_forecast_select(shape, layer.ck, forecasts, seq, B, idx, cnt, ws_s)

    want = torch.full((B, G, 18), -7, dtype=torch.int32, device=DEV), torch.zeros((B, G), dtype=torch.int32, device=DEV)
    run(*want, torch.cuda.synchronize)
    for _ in range(20):
        got = torch.full_like(want[0], -7), torch.zeros_like(want[1])
        layer.ck.fill_(NAN)
        run(*got, lambda: None)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert sb.sparda_device_error() == 0


def test_captured_and_replayed_with_other_lengths():
    G, H, B, N = 2, 16, 4, 10
    g = _gen(50)
    shape = sb.Shape(n_groups=G, heads_per_group=H, topk=8, max_ctx=8192, max_batch=B)
    layer = _layer(shape, g, [8192] * B)
    layer.ck.copy_(_randn(layer.ck.shape, g))
    start = _copy(layer)
    q, k, v = _projection((B, N), G, H, g)
    pq, pk, pv = _projection((900,), G, H, g)
    seq, nodes, path, n_path, cu = _i32([0] * B), _i32([N] * B), _i32([[0] * N] * B), _i32([0] * B), _i32([0] * (B + 1))
    parent = _i32([[-1] + [i // 2 for i in range(N - 1)]] * B)
    out, pout = torch.zeros((B, N, G * H, D), dtype=torch.bfloat16, device=DEV), torch.zeros((900, G * H, D), dtype=torch.bfloat16, device=DEV)
    ws_t, ws_p = sb.workspace(shape, B, sb.WS_TREE), sb.workspace(shape, B, sb.WS_PROMPT)
    new, new2 = _i32([0] * B), _i32([0] * B)

    def run():
        sb.sparda_prompt_attn(shape, pq, pk, pv, cu, B, pout, ws_p, past=layer, past_len=seq)
        sb.sparda_prompt_append(shape, layer, pk, pv, cu, seq, B, new_len=new)
        sb.sparda_tree_attn(shape, layer, q, k, v, parent, new, B, out, ws_t, n_nodes=nodes)
        sb.sparda_tree_commit(shape, layer, k, v, path, n_path, new, B, new_len=new2)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            run()
    for lens, past, nn in (([0, 0, 0, 0], [0, 0, 0, 0], [1, 0, 10, 3]), ([300, 200, 100, 300], [7000, 5, 64, 0], [10, 10, 2, 1]),
                           ([1, 0, 899, 0], [1, 8000, 63, 128], [10, 1, 0, 9])):
        cu.copy_(_i32([sum(lens[:i]) for i in range(B + 1)]))
        seq.copy_(_i32(past))
        nodes.copy_(_i32(nn))
        path.copy_(_i32([list(range(N))] * B))
        n_path.copy_(_i32([min(x, 3) for x in nn]))
        res = []
        for replay in (False, True):
            for x, y in ((layer.k, start.k), (layer.v, start.v), (layer.ck, start.ck)):
                x.copy_(y)
            out.fill_(7.0)
            pout.fill_(7.0)
            torch.cuda.synchronize()
            if replay:
                graph.replay()
            else:
                run()
            torch.cuda.synchronize()
            assert sb.sparda_device_error() == 0
            res.append([t.clone() for t in (pout, out, layer.k, layer.v, layer.ck, new, new2)])
        for x, y in zip(*res):
            assert torch.equal(x, y)
        assert res[0][6].tolist() == [a + b + min(c, 3) for a, b, c in zip(past, lens, nn)]


def test_calls_back_to_back_and_on_two_streams():
    """Many calls in a row that share a workspace, and two streams with workspaces of their own: the same bits."""
    G, H = 2, 16
    cases = []
    for seed, (B, N, ctx) in enumerate(((1, 1, 9000), (2, 40, 3000), (4, 8, 700), (1, 128, 2000))):
        g = _gen(60 + seed)
        shape = _shape(G, H, ctx + 64, B)
        layer = _layer(shape, g, [ctx - 7 * b for b in range(B)])
        q, k, v = _projection((B, N), G, H, g)
        cases.append((shape, layer, q, k, v, _i32([ctx - 7 * b for b in range(B)]), B, N))
    ws = [sb.workspace(cases[0][0], 1, sb.WS_TREE) for _ in range(2)]

    def run(c, w):
        shape, layer, q, k, v, seq, B, N = c
        out = torch.empty((B, N, G * H, D), dtype=torch.bfloat16, device=DEV)
        sb.sparda_tree_attn(shape, layer, q, k, v, None, seq, B, out, w)
        return out

    first = [run(c, ws[0]) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = ([], [])
    for i in range(20):
        for s, w, o in zip(streams, ws, outs):
            with torch.cuda.stream(s):
                o.append(run(cases[i % 4], w))
    torch.cuda.synchronize()
    for o in outs:
        for i, x in enumerate(o):
            assert torch.equal(x, first[i % 4])
    assert sb.sparda_device_error() == 0


def test_outputs_on_16_bytes():
    G, H, n = 1, 3, 70
    g = _gen(70)
    shape = _shape(G, H, 64, 1)
    q, k, v = _projection((n,), G, H, g)
    ws = sb.workspace(shape, 1, sb.WS_PROMPT)
    buf = torch.zeros(n * G * H * D + 8, dtype=torch.bfloat16, device=DEV)
    want = torch.empty((n, G * H, D), dtype=torch.bfloat16, device=DEV)
    off = buf[8:].view(n, G * H, D)
    assert off.data_ptr() % 32 == 16
    sb.sparda_prompt_attn(shape, q, k, v, _i32([0, n]), 1, want, ws)
    sb.sparda_prompt_attn(shape, q, k, v, _i32([0, n]), 1, off, ws)
    assert torch.equal(off, want) and bool((buf[:8] == 0).all())


def test_long_caches_beyond_32_bit_offsets():
    """The last of 66 sequences of 262144 tokens: 2^31 elements and more before it."""
    G, H, B, ctx, N = 1, 16, 66, 262144, 4
    g = _gen(80)
    shape = sb.Shape(n_groups=G, heads_per_group=H, topk=8, max_ctx=ctx, max_batch=B)
    layer = sb.LayerKV.empty(shape)
    S = [0] * (B - 1) + [ctx - 50]
    layer.k[-1].copy_(_randn(layer.k[-1].shape, g))
    layer.v[-1].copy_(_randn(layer.v[-1].shape, g))
    q, k, v = _projection((B, N), G, H, g)
    out = torch.empty((B, N, G * H, D), dtype=torch.bfloat16, device=DEV)
    sb.sparda_tree_attn(shape, layer, q, k, v, None, _i32(S), B, out, sb.workspace(shape, B, sb.WS_TREE))
    kk, vv = torch.cat((layer.k[-1, 0, : S[-1]], k[-1, :, 0])).double(), torch.cat((layer.v[-1, 0, : S[-1]], v[-1, :, 0])).double()
    on = torch.ones((N, S[-1] + N), dtype=torch.bool, device=DEV).tril(S[-1])
    for h in (0, 15):
        want, bound = attend(q[-1, :, h].double(), kk, vv, on)
        _check(out[-1, :, h], want, bound, "head %d" % h)
    sb.sparda_tree_commit(shape, layer, k, v, _i32([[0, 1, 2, 3]] * B), _i32([0] * (B - 1) + [4]), _i32(S), B)
    assert torch.equal(layer.k[-1, 0, S[-1] : S[-1] + 4], k[-1, :, 0]) and torch.equal(layer.v[-1, 0, S[-1] : S[-1] + 4], v[-1, :, 0])
    assert sb.sparda_device_error() == 0


def test_binding_refusals():
    G, H, B, N = 2, 4, 2, 5
    g = _gen(90)
    shape = _shape(G, H, 256, B)
    layer = _layer(shape, g, [10, 20])
    q, k, v = _projection((B, N), G, H, g)
    seq, out, ws = _i32([10, 20]), torch.empty((B, N, G * H, D), dtype=torch.bfloat16, device=DEV), sb.workspace(shape, B, sb.WS_TREE)

    def call(**kw):
        a = {**dict(layer=layer, q=q, k=k, v=v, parent=None, seq=seq, out=out, ws=ws), **kw}
        sb.sparda_tree_attn(shape, a["layer"], a["q"], a["k"], a["v"], a["parent"], a["seq"], B, a["out"], a["ws"],
                            n_nodes=a.get("nodes"), idx=a.get("idx"), cnt=a.get("cnt"))
    call()
    for bad in (dict(q=q[:, :, :, :64]), dict(q=q.float()), dict(q=q[:1]), dict(k=k[:, :4]), dict(v=v.transpose(0, 1)),
                dict(q=q.permute(0, 1, 3, 2)), dict(seq=seq.long()), dict(seq=seq[:1]), dict(out=out[:1]), dict(out=out.float()),
                dict(parent=_i32([[0] * N])), dict(nodes=_i32([1])), dict(idx=_i32([0])), dict(ws=ws.cpu()), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(sb.SpardaError):
        call(ws=ws[:1000])
    # every other row of twice as many: evenly spaced, but not one sequence behind the other
    wide = _projection((B, 2 * N), G, H, g)
    with pytest.raises(ValueError):
        call(q=wide[0][:, :N], k=wide[1][:, :N], v=wide[2][:, :N])
    call(q=wide[0][:, ::2], k=wide[1][:, ::2], v=wide[2][:, ::2])
    kv4 = sb.LayerKV4.empty(shape)
    with pytest.raises((ValueError, AttributeError)):
        call(layer=kv4)
