"""Measured cases of the attention of many new tokens over a bf16 cache, and of their store into it.

Operators (the formulas are in include/sparda.h beside each entry point):

  prompt   causal attention of packed prompts of different lengths, on top of what the cache
           already holds of each sequence or of nothing (sparda_prompt_attn)
  store    packed prompts' keys and values into the cache, with the compressed keys of the
           windows they complete (sparda_prompt_append)
  tree     attention of a tree of drafted tokens per sequence over the cache, over all its
           tokens or over selected blocks (sparda_tree_attn)
  commit   the accepted path of each tree into the cache, with its compressed keys
           (sparda_tree_commit)

With ``own`` false, ``run`` computes them in elementary torch operations; with ``own`` true it
calls the library.

Shapes: d = 128, blocks of 64 tokens, G KV groups of H query heads, a cache [B, G, cap, 128]. The
queries, keys and values of the new tokens are slices of one projection [tokens, G*H + 2*G, 128].
"""
import torch

own = False

D, BLOCK = 128, 64
SCALE = 1.0 / D**0.5


# ------------------------------------------------------------------------------- cases
def _case(name, op, **kw):
    # T: tokens of the longest sequence (prompt, store) or of its cache (tree, commit); past: tokens that
    # the cache holds already (prompt, store); N: nodes of a tree; topk: 0 for all tokens
    c = dict(op=op, B=1, G=2, H=16, T=1, past=0, N=0, ragged=False, topk=0)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one short chat prompt, odd length
        _case("prompt_short", "prompt", T=337),
        # a prefill batch of prompts of different lengths, packed
        _case("prompt_packed", "prompt", B=8, T=4001, ragged=True),
        # one long document
        _case("prompt_long", "prompt", T=32768),
        # the next turn of four conversations, over what their caches hold; many small KV groups
        _case("prompt_turn", "prompt", B=4, G=8, H=4, T=500, past=32768, ragged=True),
        # a short prompt into an empty cache
        _case("store_short", "store", T=1237),
        # a prefill batch of long documents into the cache
        _case("store_batch", "store", B=4, T=131072, ragged=True),
        # one user's draft over a short conversation
        _case("tree_short", "tree", T=1000, N=8),
        # a serving batch over the selected blocks of long contexts
        _case("tree_sparse_16", "tree", B=16, T=131072, N=16, topk=32, ragged=True),
        # the same batch over all tokens
        _case("tree_dense_16", "tree", B=16, T=131072, N=8),
        # large trees over a ragged batch, many small KV groups
        _case("tree_large", "tree", B=4, G=8, H=5, T=32768, N=61, ragged=True),
        # one user's accepted tokens
        _case("commit_1", "commit", T=8191, N=8),
        # a serving batch's accepted tokens
        _case("commit_64", "commit", B=64, T=4096, N=32, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    while True:
        op = rng.choice(("prompt", "prompt", "store", "tree", "tree", "commit"))
        G = rng.choice((1, 2, 2, 3, 4, 8))
        H = rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16))
        B = _log_int(rng, 1, 64)
        T = _log_int(rng, 1, 131072 if op in ("store", "tree") else 32768)
        past = _log_int(rng, 1, 65536) if op in ("prompt", "store") and rng.random() < 0.5 else 0
        N = _log_int(rng, 1, 128) if op in ("tree", "commit") else 0
        topk = rng.randint(1, 62) if op == "tree" and rng.random() < 0.5 else 0
        c = _case("", op, B=B, G=G, H=H, T=T, past=past, N=N, ragged=rng.random() < 0.7, topk=topk)
        w = work(c)
        # no larger than the largest listed ones, in work and in the caches' memory
        if w["flops"] <= 8.8e12 and w["bytes"] <= 2.2e9 and B * G * (T + past) <= 16 * 2 * 131072:
            return c


# ------------------------------------------------------------------------------- inputs
def _lens(n, ragged, B, gen):
    """Lengths: all n, or spread over [n/2, n] with one of n."""
    t = torch.full((B,), n, dtype=torch.int64)
    if ragged:
        t = n - (torch.rand(B, generator=gen) * (n // 2)).floor().to(torch.int64)
        t[0] = n
    return t.tolist()


def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _keys(shape, gen, gain, off):
    """Keys as a layer makes them: a few strong channels and channel offsets, per KV group."""
    k = torch.randn(shape, generator=gen, device="cuda")
    return k.mul_(gain).add_(off).to(torch.bfloat16)


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _window_means(k):
    """Compressed keys bf16 [B, G, W, 128] of a whole cache: means of 32 keys, every 16."""
    B, G, cap, _ = k.shape
    m = k.view(B, G, cap // 16, 16, D).float().mean(dim=3)
    return ((m[:, :, :-1] + m[:, :, 1:]) * 0.5).to(torch.bfloat16)


def _selection(B, G, topk, lens, nb, gen):
    """idx [B, G, topk+2] / cnt [B, G] as the selectors write them for the token behind the context:
    block 0, the block that token lands in and topk others, ascending, -1 behind."""
    ks = topk + 2
    tb = (_int(lens).long() // BLOCK)[:, None, None]
    j = torch.arange(nb, device="cuda")
    score = torch.rand((B, G, nb), generator=gen, device="cuda")
    score = torch.where((j == 0) | (j == tb), torch.full_like(score, 2.0), torch.where(j < tb, score, torch.full_like(score, -1.0)))
    top, at = score.topk(min(ks, nb), dim=-1)
    at = torch.where(top >= 0, at, torch.full_like(at, 1 << 30)).sort(dim=-1).values
    idx = torch.full((B, G, ks), -1, dtype=torch.int32, device="cuda")
    idx[..., : at.shape[-1]] = torch.where(at < (1 << 30), at, torch.full_like(at, -1)).to(torch.int32)
    return idx, (idx >= 0).sum(dim=-1).to(torch.int32)


def _parents(B, N, gen):
    """Trees [B, N]: node 0 is the root, every other one hangs on one of the eight nodes before it."""
    p = torch.full((B, N), -1, dtype=torch.int64)
    for i in range(1, N):
        p[:, i] = torch.randint(max(0, i - 8), i, (B,), generator=gen)
    return p.tolist()


def _paths(parents, nodes, gen):
    """The path from the root to a random node of each tree."""
    paths = []
    for par, n in zip(parents, nodes):
        at, path = int(torch.randint(0, n, (1,), generator=gen)), []
        while at >= 0:
            path.append(at)
            at = par[at]
        paths.append(path[::-1])
    return paths


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    host = torch.Generator()
    host.manual_seed(int(seed) + 1)
    op, B, G, H, N = c["op"], c["B"], c["G"], c["H"], c["N"]
    s = dict(op=op, B=B, G=G, H=H, N=N, topk=c["topk"])
    gain = 1.0 + 3.0 * (torch.rand((G, 1, D), generator=gen, device="cuda") < 0.05)
    off = 0.5 * torch.randn((G, 1, D), generator=gen, device="cuda")
    new = op in ("prompt", "store")
    # cached tokens and new tokens of every sequence
    s["ctx"] = ctx = _lens(c["past"] if new else c["T"], c["ragged"], B, host)
    if new:
        # packed rows: as many with every seed
        fixed = torch.Generator()
        fixed.manual_seed(1000 * c["T"] + B)
        lens = _lens(c["T"], c["ragged"], B, fixed)
    else:
        lens = _lens(N, c["ragged"], B, host)
    s["lens"] = lens
    room = max(x + y for x, y in zip(ctx, lens)) + (0 if new else N)
    s["cap"] = cap = (room + BLOCK - 1) // BLOCK * BLOCK
    s["ctx_dev"] = _int(ctx)
    if op != "prompt" or c["past"]:
        s["k"], s["v"] = _keys((B, G, cap, D), gen, gain, off), _randn((B, G, cap, D), gen)
    if op in ("store", "commit"):
        s["ck"] = _window_means(s["k"])
    # the new tokens' projection: queries, keys and values of a token beside one another
    rows = sum(lens) if new else B * N
    qkv = torch.empty((rows, G * H + 2 * G, D), dtype=torch.bfloat16, device="cuda")
    qkv[:, : G * H] = _randn((rows, G * H, D), gen)
    qkv[:, G * H : G * H + G] = _keys((rows, G, D), gen, gain[:, 0], off[:, 0])
    qkv[:, G * H + G :] = _randn((rows, G, D), gen)
    if not new:
        qkv = qkv.view(B, N, G * H + 2 * G, D)
        parents = _parents(B, N, host)
        s["parents"], s["parent"], s["nodes"] = parents, _int(parents), _int(lens)
    s["q"], s["k_new"], s["v_new"] = qkv[..., : G * H, :], qkv[..., G * H : G * H + G, :], qkv[..., G * H + G :, :]
    if new:
        s["cu"] = _int([sum(lens[:i]) for i in range(B + 1)])
    if op in ("prompt", "tree"):
        s["out"] = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    if op == "tree" and c["topk"]:
        s["idx"], s["cnt"] = _selection(B, G, c["topk"], ctx, cap // BLOCK, gen)
    if op == "commit":
        s["paths"] = paths = _paths(parents, lens, host)
        s["path"] = _int([p + [-1] * (N - len(p)) for p in paths])
        s["n_path"] = _int([len(p) for p in paths])
    if op in ("store", "commit"):
        s["new_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if own:
        _own_state(s)
    return s


def _own_state(s):
    """The library's handles: shape, layer, workspace."""
    import block_sparse_attention_forecast_gb300.binding as sb

    s["sb"] = sb
    B, G, op = s["B"], s["G"], s["op"]
    s["shape"] = shape = sb.Shape(n_groups=G, heads_per_group=s["H"], topk=max(1, s["topk"]), max_ctx=s["cap"], max_batch=B)
    s["layer"] = None
    if "k" in s:
        ck = s["ck"] if "ck" in s else torch.zeros((B, G, max(0, s["cap"] // 16 - 1), D), dtype=torch.bfloat16, device="cuda")
        s["layer"] = sb.LayerKV(s["k"], s["v"], ck)
    if op in ("prompt", "tree"):
        s["ws"] = sb.workspace(shape, B, sb.WS_PROMPT if op == "prompt" else sb.WS_TREE)


# ------------------------------------------------------------------------------- one pass
def run(state):
    s = state
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    sb, shape, layer, B, op = s["sb"], s["shape"], s["layer"], s["B"], s["op"]
    if op == "prompt":
        past = dict(past=layer, past_len=s["ctx_dev"]) if layer is not None else {}
        sb.sparda_prompt_attn(shape, s["q"], s["k_new"], s["v_new"], s["cu"], B, s["out"], s["ws"], **past)
        return dict(out=s["out"])
    if op == "tree":
        sb.sparda_tree_attn(shape, layer, s["q"], s["k_new"], s["v_new"], s["parent"], s["ctx_dev"], B, s["out"], s["ws"],
                            n_nodes=s["nodes"], idx=s.get("idx"), cnt=s.get("cnt"))
        return dict(out=s["out"])
    if op == "store":
        sb.sparda_prompt_append(shape, layer, s["k_new"], s["v_new"], s["cu"], s["ctx_dev"], B, new_len=s["new_len"])
    else:
        sb.sparda_tree_commit(shape, layer, s["k_new"], s["v_new"], s["path"], s["n_path"], s["ctx_dev"], B,
                              new_len=s["new_len"])
    return dict(k=layer.k, v=layer.v, ck=layer.ck, new_len=s["new_len"])


def _softmax_values(sc, v):
    """softmax(sc) v in 32 bits; sc [.., n], -inf where a key is not attended."""
    p = torch.exp(sc - sc.amax(dim=-1, keepdim=True))
    return torch.matmul(p, v) / p.sum(dim=-1, keepdim=True)


def _run_plain(s):
    op = s["op"]
    if op == "prompt":
        return _prompt_plain(s)
    if op == "tree":
        return _tree_plain(s)
    return _store_plain(s)


def _prompt_plain(s):
    G, H, out, first = s["G"], s["H"], s["out"], 0
    for b, (P, n) in enumerate(zip(s["ctx"], s["lens"])):
        k, v = s["k_new"][first : first + n].transpose(0, 1), s["v_new"][first : first + n].transpose(0, 1)
        if P:
            k, v = torch.cat((s["k"][b, :, :P], k), dim=1), torch.cat((s["v"][b, :, :P], v), dim=1)
        k, v = k.float(), v.float()
        # as many rows at once as 2^28 scores allow
        step = max(1, (1 << 28) // (G * H * (P + n)))
        for i in range(0, n, step):
            m = min(step, n - i)
            q = s["q"][first + i : first + i + m].float().view(m, G, H, D).permute(1, 2, 0, 3)
            end = P + i + m
            sc = torch.matmul(q.reshape(G, H * m, D), k[:, :end].transpose(1, 2)).mul_(SCALE).view(G, H, m, end)
            row = P + i + torch.arange(m, device="cuda")
            sc.masked_fill_(torch.arange(end, device="cuda")[None] > row[:, None], float("-inf"))
            o = _softmax_values(sc.view(G, H * m, end), v[:, :end]).view(G, H, m, D)
            out[first + i : first + i + m] = o.permute(2, 0, 1, 3).reshape(m, G * H, D).to(torch.bfloat16)
        first += n
    return dict(out=out)


def _tree_plain(s):
    G, H, N, out = s["G"], s["H"], s["N"], s["out"]
    # sees[b, i, j]: node j is node i or an ancestor of it
    B = s["B"]
    eye = torch.eye(N, dtype=torch.bool, device="cuda")
    sees = eye.expand(B, N, N).clone()
    at = s["parent"].long()
    for _ in range(N):
        sees |= torch.nn.functional.one_hot(at.clamp(min=0), N).bool() & (at >= 0)[..., None]
        at = torch.where(at >= 0, s["parent"].long().gather(1, at.clamp(min=0)), at)
    for b, (S, n) in enumerate(zip(s["ctx"], s["lens"])):
        if s["topk"]:
            idx = s["idx"][b].long()
            pos = (idx.clamp(min=0)[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(1)
            ok = (pos < S) & (idx >= 0).repeat_interleave(BLOCK, dim=1)
            g = torch.arange(G, device="cuda")[:, None]
            k, v = s["k"][b][g, pos], s["v"][b][g, pos]
        else:
            k, v = s["k"][b, :, :S], s["v"][b, :, :S]
            ok = torch.ones((G, S), dtype=torch.bool, device="cuda")
        m = ok.shape[1]
        k = torch.cat((k, s["k_new"][b, :n].transpose(0, 1)), dim=1).float()
        v = torch.cat((v, s["v_new"][b, :n].transpose(0, 1)), dim=1).float()
        q = s["q"][b, :n].float().view(n, G, H, D).permute(1, 0, 2, 3)
        sc = torch.matmul(q.reshape(G, n * H, D), k.transpose(1, 2)).mul_(SCALE).view(G, n, H, m + n)
        on = torch.cat((ok[:, None, None].expand(G, n, 1, m), sees[b, :n, :n][None, :, None].expand(G, n, 1, n)), dim=-1)
        sc.masked_fill_(~on, float("-inf"))
        o = _softmax_values(sc.view(G, n * H, m + n), v).view(G, n, H, D)
        out[b, :n] = o.permute(1, 0, 2, 3).reshape(n, G * H, D).to(torch.bfloat16)
    return dict(out=out)


def _store_plain(s):
    first = 0
    for b, S in enumerate(s["ctx"]):
        if s["op"] == "store":
            n = s["lens"][b]
            k, v = s["k_new"][first : first + n], s["v_new"][first : first + n]
            first += n
        else:
            n = len(s["paths"][b])
            at = s["path"][b, :n].long()
            k, v = s["k_new"][b][at], s["v_new"][b][at]
        s["k"][b, :, S : S + n] = k.transpose(0, 1)
        s["v"][b, :, S : S + n] = v.transpose(0, 1)
        # the windows that the new tokens complete: window w is keys 16w .. 16w+31
        w0, w1 = max(0, (S - 16) // 16), max(0, (S + n - 16) // 16)
        if w1 > w0:
            x = s["k"][b, :, 16 * w0 : 16 * w1 + 16].double().unflatten(1, (w1 - w0 + 1, 16)).sum(dim=2)
            s["ck"][b, :, w0:w1] = ((x[:, :-1] + x[:, 1:]) / 32.0).to(torch.bfloat16)
        s["new_len"][b] = S + n
    return dict(k=s["k"], v=s["v"], ck=s["ck"], new_len=s["new_len"])


# ------------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    B, G, H, T, N, op, past = c["B"], c["G"], c["H"], c["T"], c["N"], c["op"], c["past"]
    row = 2 * D

    def mean(n):
        return n - (n // 2) / 2.0 * (B - 1) / B if c["ragged"] else float(n)

    t = mean(T)
    if op == "prompt":
        p = mean(past)
        # (query, key) pairs of one sequence: the past and the tokens up to its own
        pairs = t * p + t * (t + 1) / 2.0
        return dict(bytes=B * G * (2 * H * t * row + 2 * t * row + 2 * p * row), flops=4.0 * D * B * G * H * pairs)
    if op == "store":
        # rows in, rows out, and the compressed keys
        return dict(bytes=B * G * t * (4 * row + row / 16.0), flops=B * G * t * 2 * D)
    n = mean(N)
    if op == "commit":
        # about half of a deep tree's nodes at most are accepted; the keys of a window that reaches back
        return dict(bytes=B * G * (n / 4.0 * 4 * row + 16 * row), flops=B * G * 32 * D)
    tokens = min(t, (c["topk"] + 2) * BLOCK) if c["topk"] else t
    return dict(bytes=B * G * (2 * tokens * row + 2 * n * row + 2 * H * n * row), flops=4.0 * D * B * G * H * n * (tokens + n / 2.0))


# ------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The same outputs from the definitions in 64 bits, one KV group at a time."""
    global own
    if work(case)["flops"] > 1.0e13:
        return None
    kept_own, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept_own
    op, G, H = s["op"], s["G"], s["H"]
    if op in ("store", "commit"):
        return dict(k=None, v=None, ck=_exact_windows(s), new_len=None)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for b in range(s["B"]):
        n, S = s["lens"][b], s["ctx"][b]
        if op == "prompt":
            q, kn, vn, o = (x[first : first + n] for x in (s["q"], s["k_new"], s["v_new"], out))
            first += n
        else:
            q, kn, vn, o = s["q"][b, :n], s["k_new"][b, :n], s["v_new"][b, :n], out[b, :n]
        if op == "tree":
            line = torch.zeros((n, n), dtype=torch.bool)
            for i in range(n):
                j = i
                while j >= 0:
                    line[i, j] = True
                    j = s["parents"][b][j]
            line = line.cuda()
        for g in range(G):
            on = None
            if "k" not in s or S == 0:
                kc = vc = torch.zeros((0, D), dtype=torch.float64, device="cuda")
            elif "idx" in s:
                hit = torch.zeros(s["cap"] // BLOCK, dtype=torch.bool, device="cuda")
                hit[s["idx"][b, g, : int(s["cnt"][b, g])].long()] = True
                t = torch.arange(S, device="cuda")
                t = t[hit[t // BLOCK]]
                kc, vc = s["k"][b, g, t].double(), s["v"][b, g, t].double()
            else:
                kc, vc = s["k"][b, g, :S].double(), s["v"][b, g, :S].double()
            m = kc.shape[0]
            kk, vv = torch.cat((kc, kn[:, g].double())), torch.cat((vc, vn[:, g].double()))
            step = max(1, (1 << 26) // (H * (m + n)))
            for i in range(0, n, step):
                e = min(n, i + step)
                last = m + (e if op == "prompt" else n)
                z = torch.einsum("thc,uc->thu", q[i:e, g * H : g * H + H].double(), kk[:last]) / D**0.5
                if op == "prompt":
                    on = torch.ones((e - i, last), dtype=torch.bool, device="cuda").tril(m + i)
                else:
                    on = torch.cat((torch.ones((e - i, m), dtype=torch.bool, device="cuda"), line[i:e]), dim=1)
                z = torch.where(on[:, None], z, torch.full((), -torch.inf, dtype=torch.float64, device="cuda"))
                z = torch.exp(z - torch.logsumexp(z, dim=-1, keepdim=True))
                o[i:e, g * H : g * H + H] = torch.einsum("thu,uc->thc", z, vv[:last])
    return dict(out=out)


def _exact_windows(s):
    """Compressed keys after the store: the mean of each completed window's 32 keys."""
    ck = s["ck"].double()
    first = 0
    for b, S in enumerate(s["ctx"]):
        if s["op"] == "store":
            new = s["k_new"][first : first + s["lens"][b]]
            first += s["lens"][b]
        else:
            new = s["k_new"][b][torch.tensor(s["paths"][b], device="cuda")]
        ends = [t for t in range(32, S + new.shape[0] + 1, 16) if t > S]
        if not ends:
            continue
        keys = torch.cat((s["k"][b, :, : S], new.transpose(0, 1)), dim=1)
        at = torch.tensor(ends, device="cuda")
        for part in at.split(1024):
            rows = (part - 32)[:, None] + torch.arange(32, device="cuda")
            ck[b, :, (part - 32) // 16] = keys[:, rows].double().mean(dim=2)
    return ck
