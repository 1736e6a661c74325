"""Measured cases of the 4-bit KV cache and of the eviction of cache blocks by attention mass.

Operators (the formulas are in include/sparda.h beside each entry point):

  prompt   a prompt's keys and values into the 4-bit cache, and the values it then holds back
           as bf16 (sparda_kv4_quantize, sparda_kv4_dequantize)
  append   one decode token into the 4-bit cache with its compressed key, and the block it
           landed in (sparda_kv4_append, sparda_kv4_dequantize of one block)
  attend   decode attention over the 4-bit cache, over the selected blocks or over all of them
           (sparda_kv4_decode_attn)
  mass     decode attention that also adds up the attention weight each block received, over
           the 4-bit or the bf16 cache (sparda_kv4_decode_attn, sparda_sparse_decode_attn_mass)
  evict    the blocks with the most accumulated weight kept and moved together into a smaller
           cache (sparda_evict_blocks, sparda_kv4_evict_blocks)

With ``own`` false, ``run`` computes them in elementary torch operations; with ``own`` true it
calls the library.

Shapes: d = 128, blocks of 64 tokens, G KV groups of H query heads. A row's 128 channels form
four groups of 32, each with its own 16-level grid: value(c) = round(scale * (16 + c) + zero).
"""
import torch

own = False

D, BLOCK, GROUP = 128, 64, 32


# ------------------------------------------------------------------------------- cases
def _case(name, op, **kw):
    c = dict(op=op, fmt="kv4", B=1, G=2, H=16, T=1, ragged=False, topk=32, keep=0, recent=0)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a short chat prompt, odd length
        _case("prompt_short", "prompt", B=1, T=1237),
        # prefill of four long documents
        _case("prompt_long", "prompt", B=4, T=131072, ragged=True),
        # a decode step's append for one long conversation, on a token that completes a window
        _case("append_1", "append", B=1, T=131072),
        # a serving batch
        _case("append_64", "append", B=64, T=16384, ragged=True),
        # one layer of a single user's decode step over the selected blocks
        _case("attend_sparse_1", "attend", B=1, T=131072),
        # one layer of the benchmark's decode step: batch 16, context 131072, top-32
        _case("attend_sparse_16", "attend", B=16, T=131072),
        # all blocks of a ragged batch, a model with many small KV groups
        _case("attend_dense_ragged", "attend", B=8, G=8, H=4, T=8191, ragged=True, topk=0),
        # all blocks of the benchmark's batch
        _case("attend_dense_16", "attend", B=16, T=131072, topk=0),
        # the decode steps between two evictions, 4-bit cache
        _case("mass_kv4_16", "mass", B=16, T=131072),
        # the same over the bf16 cache
        _case("mass_bf16_16", "mass", fmt="bf16", B=16, T=131072),
        # a long prompt cut down to 32K tokens before decode, bf16 cache
        _case("evict_bf16_4", "evict", fmt="bf16", B=4, T=131072, ragged=True, keep=512, recent=16),
        # a batch of conversations cut to 8K tokens, 4-bit cache, then unpacked for the next turn's prefill
        _case("evict_kv4_16", "evict", B=16, T=32768, ragged=True, keep=128, recent=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("prompt", "append", "attend", "attend", "mass", "evict"))
    fmt = "bf16" if op in ("mass", "evict") and rng.random() < 0.5 else "kv4"
    H = 16 if fmt == "bf16" else rng.choice((1, 2, 4, 5, 8, 12, 16))
    G = rng.choice((1, 2, 2, 3, 4, 8))
    # tokens of all sequence-groups together: at most those of the largest listed case of the operator
    cap = 4 * 2 * 131072 if op in ("prompt", "evict") else 16 * 2 * 131072
    B = _log_int(rng, 1, 64)
    T = _log_int(rng, 1, max(2, min(131072, cap // (B * G))))
    dense = op == "attend" and rng.random() < 0.5
    topk = 0 if dense else rng.randint(1, 62)
    keep = recent = 0
    if op == "evict":
        recent = _log_int(rng, 1, 24)
        keep = recent + 1 + _log_int(rng, 1, max(2, (T // BLOCK) * 2 // 3))
    return _case("", op, fmt=fmt, B=B, G=G, H=H, T=T, ragged=rng.random() < 0.7, topk=topk, keep=keep, recent=recent)


# ------------------------------------------------------------------------------- inputs
def _seq_lens(c, gen):
    """Sequence lengths: all T, or spread over [T/2, T] with one of T."""
    B, T = c["B"], c["T"]
    t = torch.full((B,), T, dtype=torch.int32, device="cuda")
    if c["ragged"]:
        r = torch.rand(B, generator=gen, device="cuda")
        t = (T - (r * (T // 2)).floor()).to(torch.int32)
        t[0] = T
    return t


def _randn(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _kv(c, gen, cap):
    """Keys and values as a layer makes them: keys with a few strong channels and channel offsets."""
    B, G = c["B"], c["G"]
    gain = 1.0 + 3.0 * (torch.rand((1, G, 1, D), generator=gen, device="cuda") < 0.05)
    off = 0.5 * torch.randn((1, G, 1, D), generator=gen, device="cuda")
    k = torch.randn((B, G, cap, D), generator=gen, device="cuda")
    k = k.mul_(gain).add_(off).to(torch.bfloat16)
    return k, _randn((B, G, cap, D), gen)


def _selection(c, gen, seq, nb):
    """idx [B, G, topk+2] / cnt [B, G] as the selectors write them: block 0, the tail block and
    topk others, ascending, -1 behind."""
    B, G, ks = c["B"], c["G"], c["topk"] + 2
    tb = ((seq.long() - 1) // BLOCK)[:, None, None]
    j = torch.arange(nb, device="cuda")
    score = torch.rand((B, G, nb), generator=gen, device="cuda")
    score = torch.where((j == 0) | (j == tb), torch.full_like(score, 2.0), torch.where(j < tb, score, torch.full_like(score, -1.0)))
    top, at = score.topk(min(ks, nb), dim=-1)
    at = torch.where(top >= 0, at, torch.full_like(at, 1 << 30)).sort(dim=-1).values
    idx = torch.full((B, G, ks), -1, dtype=torch.int32, device="cuda")
    idx[..., : at.shape[-1]] = torch.where(at < (1 << 30), at, torch.full_like(at, -1)).to(torch.int32)
    return idx, (idx >= 0).sum(dim=-1).to(torch.int32)


def _window_means(k):
    """Compressed keys bf16 [B, G, W, 128] of a whole cache: means of 32 keys, every 16."""
    B, G, cap, _ = k.shape
    m = k.view(B, G, cap // 16, 16, D).float().mean(dim=3)
    return ((m[:, :, :-1] + m[:, :, 1:]) * 0.5).to(torch.bfloat16)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, fmt, B, G, H = c["op"], c["fmt"], c["B"], c["G"], c["H"]
    nb = (c["T"] - 1) // BLOCK + 1
    cap = nb * BLOCK
    s = dict(op=op, fmt=fmt, B=B, G=G, H=H, nb=nb, cap=cap, topk=c["topk"], dense=c["topk"] == 0, keep=c["keep"],
             recent=c["recent"])
    s["seq"] = seq = _seq_lens(c, gen)
    s["k"], s["v"] = _kv(c, gen, cap)
    if op == "append":
        s["k_new"], s["v_new"] = _randn((B, G, D), gen), _randn((B, G, D), gen)
        # the block that the new token lands in, as a selection of one block
        s["topk"] = 1
        s["idx"] = torch.full((B, G, 3), -1, dtype=torch.int32, device="cuda")
        s["idx"][..., 0] = ((seq - 1) // BLOCK)[:, None]
        s["cnt"] = torch.ones((B, G), dtype=torch.int32, device="cuda")
    if op in ("attend", "mass"):
        s["q"] = _randn((B, G * H, D), gen)
        if not s["dense"]:
            s["idx"], s["cnt"] = _selection(c, gen, seq, nb)
    if op in ("mass", "evict"):
        # weights received so far: heavy-tailed, and nothing yet for blocks that were never selected
        m = torch.exp(1.5 * torch.randn((B, G, nb), generator=gen, device="cuda"))
        s["mass"] = m * (torch.rand((B, G, nb), generator=gen, device="cuda") < 0.7)
    if op in ("append", "evict"):
        s["ck"] = _window_means(s["k"])
    if op == "evict":
        dcap = c["keep"] * BLOCK
        s["kept"] = torch.zeros((B, G, c["keep"]), dtype=torch.int32, device="cuda")
        s["dst_seq"] = torch.zeros((B,), dtype=torch.int32, device="cuda")
        s["dst_mass"] = torch.zeros((B, G, c["keep"]), device="cuda")
        s["dst_ck"] = torch.zeros((B, G, dcap // 16 - 1, D), dtype=torch.bfloat16, device="cuda")
        s["dst_k"] = torch.zeros((B, G, dcap, D), dtype=torch.bfloat16, device="cuda")
        s["dst_v"] = torch.zeros_like(s["dst_k"])
    if op == "append":
        s["out_k"] = torch.zeros((B, G, 3, BLOCK, D), dtype=torch.bfloat16, device="cuda")
        s["out_v"] = torch.zeros_like(s["out_k"])
    if op == "prompt":
        s["out_k"], s["out_v"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    if own:
        _own_state(s)
    elif fmt == "kv4" and op != "prompt":
        s["qk"], s["qv"] = _quantize(s["k"], torch.bfloat16), _quantize(s["v"], torch.float16)
        del s["k"], s["v"]
    return s


def _own_state(s):
    """The library's handles: shapes, the layer's cache filled from the prompt, workspaces."""
    import block_sparse_attention_forecast_gb300.binding as sb

    s["sb"] = sb
    B, G, fmt, op = s["B"], s["G"], s["fmt"], s["op"]
    s["shape"] = shape = sb.Shape(n_groups=G, heads_per_group=s["H"], topk=max(1, s["topk"]), max_ctx=s["cap"], max_batch=B)
    s["out"] = torch.empty((B, G * s["H"], D), dtype=torch.bfloat16, device="cuda")
    if fmt == "bf16":
        ck = s["ck"] if "ck" in s else torch.zeros((B, G, max(0, s["cap"] // 16 - 1), D), dtype=torch.bfloat16, device="cuda")
        s["layer"] = sb.LayerKV(s["k"], s["v"], ck)
        s["ws"] = sb.workspace(shape, B, sb.WS_ATTN_MASS)
    else:
        s["layer"] = layer = sb.LayerKV4.empty(shape)
        if op != "prompt":
            sb.sparda_kv4_quantize(shape, layer, s["k"], s["v"], s["seq"], B)
            del s["k"], s["v"]
        if "ck" in s:
            layer.ck = s["ck"]
        s["ws"] = sb.workspace(shape, B, sb.WS_KV4_ATTN_MASS if op == "mass" else sb.WS_KV4_ATTN)
    if op == "evict":
        s["dst_shape"] = dshape = sb.Shape(n_groups=G, heads_per_group=s["H"], max_ctx=s["keep"] * BLOCK, max_batch=B)
        if fmt == "bf16":
            s["dst"] = sb.LayerKV(s["dst_k"], s["dst_v"], s["dst_ck"])
        else:
            s["dst"] = sb.LayerKV4.empty(dshape)
            s["dst"].ck = s["dst_ck"]


# ------------------------------------------------------------------------------- one pass
def run(state):
    s = state
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    sb, shape, layer, seq, B = s["sb"], s["shape"], s["layer"], s["seq"], s["B"]
    op = s["op"]
    if op == "prompt":
        sb.sparda_kv4_quantize(shape, layer, s["k"], s["v"], seq, B)
        sb.sparda_kv4_dequantize(shape, layer, seq, B, s["out_k"], s["out_v"])
        return dict(k=s["out_k"], v=s["out_v"])
    if op == "append":
        sb.sparda_kv4_append(shape, layer, s["k_new"], s["v_new"], seq, B)
        sb.sparda_kv4_dequantize(shape, layer, seq, B, s["out_k"], s["out_v"], idx=s["idx"], cnt=s["cnt"])
        return dict(k=s["out_k"], v=s["out_v"], ck=layer.ck)
    if op == "attend":
        sb.sparda_kv4_decode_attn(shape, layer, s["q"], s.get("idx"), s.get("cnt"), seq, B, s["out"], s["ws"])
        return dict(out=s["out"])
    if op == "mass":
        if s["fmt"] == "kv4":
            sb.sparda_kv4_decode_attn(shape, layer, s["q"], s["idx"], s["cnt"], seq, B, s["out"], s["ws"], mass=s["mass"])
        else:
            sb.sparda_sparse_decode_attn_mass(shape, layer, s["q"], s["idx"], s["cnt"], seq, B, s["out"], s["ws"], s["mass"])
        return dict(out=s["out"], mass=s["mass"])
    evict = sb.sparda_kv4_evict_blocks if s["fmt"] == "kv4" else sb.sparda_evict_blocks
    evict(shape, layer, s["mass"], seq, B, s["keep"], s["recent"], s["kept"], dst_shape=s["dst_shape"], dst=s["dst"],
          dst_mass=s["dst_mass"], dst_seq_len=s["dst_seq"])
    if s["fmt"] == "kv4":
        sb.sparda_kv4_dequantize(s["dst_shape"], s["dst"], s["dst_seq"], B, s["dst_k"], s["dst_v"])
    return dict(k=s["dst_k"], v=s["dst_v"], ck=s["dst_ck"], kept=s["kept"], mass=s["dst_mass"], seq_len=s["dst_seq"])


# -- the plain form: the 4-bit grid, two channels per byte
def _quantize(x, dtype):
    """x [..., 128] -> (codes packed two per byte [..., 64], scale [..., 4], zero [..., 4])."""
    g = x.float().unflatten(-1, (D // GROUP, GROUP))
    lo, hi = g.amin(dim=-1), g.amax(dim=-1)
    scale = ((hi - lo) / 15.0).to(dtype)
    zero = (lo - 16.0 * scale.float()).to(dtype)
    sf, zf = scale.float()[..., None], zero.float()[..., None]
    code = ((g - zf) / torch.where(sf > 0, sf, torch.ones_like(sf)) - 16.0).round().clamp(0, 15)
    code = torch.where(sf > 0, code, torch.zeros_like(code)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale, zero


def _values(packed, dtype):
    """The values that (codes, scale, zero) stand for, as float32."""
    codes, scale, zero = packed
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).float().unflatten(-1, (D // GROUP, GROUP))
    # scale * (16 + c) is exact in 32 bits (8 or 11 bits times 5); the sum with zero is taken in
    # 64 bits and rounded once, to the storage type
    v = (scale.float()[..., None] * (16.0 + c)).double().add_(zero.double()[..., None])
    return v.to(dtype).float().flatten(-2)


def _k_values(s):
    return _values(s["qk"], torch.bfloat16) if s["fmt"] == "kv4" else s["k"].float()


def _v_values(s):
    return _values(s["qv"], torch.float16) if s["fmt"] == "kv4" else s["v"].float()


def _gather_blocks(x, idx):
    """x [B, G, nb * 64, ...] -> [B, G, n, 64, ...], the blocks idx [B, G, n] (clamped to 0)."""
    B, G, n = idx.shape
    b = torch.arange(B, device=x.device)[:, None, None]
    g = torch.arange(G, device=x.device)[None, :, None]
    return x.unflatten(2, (-1, BLOCK))[b, g, idx.long().clamp(min=0)]


def _select(s):
    """The cache entries that the attention reads, float32 [B, G, n, 64, 128], their validity, and the blocks."""
    B, G, nb = s["B"], s["G"], s["nb"]
    if s["dense"]:
        idx = torch.arange(nb, device="cuda").expand(B, G, nb)
        k, v = _k_values(s).unflatten(2, (nb, BLOCK)), _v_values(s).unflatten(2, (nb, BLOCK))
    else:
        idx = s["idx"].long()
        if s["fmt"] == "kv4":
            k = _values([_gather_blocks(x, idx) for x in s["qk"]], torch.bfloat16)
            v = _values([_gather_blocks(x, idx) for x in s["qv"]], torch.float16)
        else:
            k, v = _gather_blocks(s["k"], idx).float(), _gather_blocks(s["v"], idx).float()
    pos = idx[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")
    ok = (pos < s["seq"].long()[:, None, None, None]) & (idx >= 0)[..., None]
    return k, v, ok, idx


def _attend(s):
    """(out, weights [B, G, n] that each block received over the group's heads)."""
    B, G, H = s["B"], s["G"], s["H"]
    k, v, ok, idx = _select(s)
    n = idx.shape[2]
    q = s["q"].float().view(B, G, H, D)
    sc = torch.matmul(q, k.flatten(2, 3).transpose(-1, -2)) * (1.0 / D**0.5)
    sc = sc.masked_fill(~ok.flatten(2)[:, :, None, :], float("-inf"))
    p = torch.exp(sc - sc.amax(dim=-1, keepdim=True))
    p = p / p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p, v.flatten(2, 3))
    w = p.unflatten(-1, (n, BLOCK)).sum(dim=(2, 4))
    return out.to(torch.bfloat16).view(B, G * H, D), w


def _run_plain(s):
    op, B, G = s["op"], s["B"], s["G"]
    if op == "prompt":
        live = torch.arange(s["cap"], device="cuda") < s["seq"].long()[:, None]
        live = live[:, None, :, None]
        k = _values(_quantize(s["k"], torch.bfloat16), torch.bfloat16).to(torch.bfloat16)
        v = _values(_quantize(s["v"], torch.float16), torch.float16).to(torch.bfloat16)
        s["out_k"].copy_(torch.where(live, k, s["out_k"]))
        s["out_v"].copy_(torch.where(live, v, s["out_v"]))
        return dict(k=s["out_k"], v=s["out_v"])
    if op == "append":
        return _append_plain(s)
    if op in ("attend", "mass"):
        out, w = _attend(s)
        if op == "attend":
            return dict(out=out)
        w = torch.where(s["idx"] >= 0, w, torch.zeros_like(w))
        s["mass"].scatter_add_(2, s["idx"].long().clamp(min=0), w)
        return dict(out=out, mass=s["mass"])
    return _evict_plain(s)


def _append_plain(s):
    B, G, seq = s["B"], s["G"], s["seq"].long()
    b = torch.arange(B, device="cuda")[:, None]
    g = torch.arange(G, device="cuda")[None, :]
    at = (seq - 1)[:, None].expand(B, G)
    for cache, new, dtype in ((s["qk"], s["k_new"], torch.bfloat16), (s["qv"], s["v_new"], torch.float16)):
        for held, put in zip(cache, _quantize(new, dtype)):
            held[b, g, at] = put
    # the compressed key of the window that the token completes
    if s["ck"].shape[2]:
        i = ((seq - 32) // 16).clamp(min=0)
        rows = (16 * i)[:, None] + torch.arange(32, device="cuda")
        rows = rows.clamp(max=s["cap"] - 1)
        win = _values([x[b[..., None], g[..., None], rows[:, None, :]] for x in s["qk"]], torch.bfloat16)
        mean = win.double().mean(dim=2).to(torch.bfloat16)
        done = ((seq >= 32) & ((seq - 32) % 16 == 0))[:, None, None]
        old = s["ck"][b, g, i[:, None].expand(B, G)]
        s["ck"][b, g, i[:, None].expand(B, G)] = torch.where(done, mean, old)
    # the block it landed in
    live = (s["idx"][:, :, :1, None].long() * BLOCK + torch.arange(BLOCK, device="cuda")) < seq[:, None, None, None]
    for name, cache, dtype in (("out_k", s["qk"], torch.bfloat16), ("out_v", s["qv"], torch.float16)):
        x = _values([_gather_blocks(t, s["idx"][..., :1]) for t in cache], dtype).to(torch.bfloat16)
        s[name][:, :, :1] = torch.where(live[..., None], x, s[name][:, :, :1])
    return dict(k=s["out_k"], v=s["out_v"], ck=s["ck"])


def _kept_blocks(s):
    """(kept [B, G, keep] old block numbers, ascending, -1 behind; count [B]; blocks before [B])."""
    B, G, nb, keep, recent = s["B"], s["G"], s["nb"], s["keep"], s["recent"]
    n = (s["seq"].long() - 1) // BLOCK + 1
    j = torch.arange(nb, device="cuda")
    n3 = n[:, None, None]
    forced = (j == 0) | ((j >= n3 - recent) & (j < n3))
    key = torch.where(forced, torch.full_like(s["mass"], float("inf")), s["mass"])
    key = torch.where(j < n3, key, torch.full_like(key, float("-inf")))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    order = torch.where(order < n3, order, torch.full_like(order, 1 << 30)).sort(dim=-1).values
    kept = torch.full((B, G, keep), -1, dtype=torch.int64, device="cuda")
    kept[..., : order.shape[-1]] = torch.where(order < (1 << 30), order, torch.full_like(order, -1))
    return kept, n.clamp(max=keep), n


def _evict_plain(s):
    B, G, keep, nb = s["B"], s["G"], s["keep"], s["nb"]
    kept, count, n = _kept_blocks(s)
    new_len = s["seq"].long() - BLOCK * (n - count)
    live = (kept >= 0)[..., None, None]
    if s["fmt"] == "kv4":
        k = _values([_gather_blocks(x, kept) for x in s["qk"]], torch.bfloat16).to(torch.bfloat16)
        v = _values([_gather_blocks(x, kept) for x in s["qv"]], torch.float16).to(torch.bfloat16)
        pos = (torch.arange(keep, device="cuda") * BLOCK)[:, None] + torch.arange(BLOCK, device="cuda")
        live_out = (pos < new_len[:, None, None, None])[..., None]
    else:
        k, v = _gather_blocks(s["k"], kept), _gather_blocks(s["v"], kept)
        live_out = live
    dk, dv = s["dst_k"].unflatten(2, (keep, BLOCK)), s["dst_v"].unflatten(2, (keep, BLOCK))
    s["dst_k"] = torch.where(live_out, k, dk).flatten(2, 3)
    s["dst_v"] = torch.where(live_out, v, dv).flatten(2, 3)
    s["kept"].copy_(kept)
    s["dst_seq"].copy_(new_len)
    mass = s["mass"].gather(2, kept.clamp(min=0))
    s["dst_mass"].copy_(torch.where(kept >= 0, mass, torch.zeros_like(mass)))
    # compressed keys: windows 4j .. 4j+3 start in block j; the last of them reaches into the next
    # block, so it is formed anew where that one is not the old neighbour
    if s["dst_ck"].shape[2]:
        old = torch.nn.functional.pad(s["ck"], (0, 0, 0, 1)).unflatten(2, (nb, 4))
        b = torch.arange(B, device="cuda")[:, None, None]
        g = torch.arange(G, device="cuda")[None, :, None]
        ck = old[b, g, kept.clamp(min=0)]
        nxt = torch.cat((kept[..., 1:], kept[..., -1:]), dim=-1)
        span = torch.cat((k[:, :, :, 48:], torch.roll(k, -1, dims=2)[:, :, :, :16]), dim=3)
        joined = span.double().mean(dim=3).to(torch.bfloat16)
        ck[:, :, :, 3] = torch.where((nxt == kept + 1)[..., None], ck[:, :, :, 3], joined)
        ck = ck.flatten(2, 3)[:, :, : 4 * keep - 1]
        windows = ((new_len - 32) // 16 + 1).clamp(min=0)
        done = torch.arange(4 * keep - 1, device="cuda") < windows[:, None]
        s["dst_ck"].copy_(torch.where(done[:, None, :, None], ck, s["dst_ck"]))
    return dict(k=s["dst_k"], v=s["dst_v"], ck=s["dst_ck"], kept=s["kept"], mass=s["dst_mass"], seq_len=s["dst_seq"])


# ------------------------------------------------------------------------------- what a pass cannot do without
KV4_ROW = 64 + 16          # 128 codes of 4 bits, four (scale, zero) pairs of 2 x 16 bits
BF16_ROW = 2 * D


def work(case):
    c = case
    B, G, H, T, op = c["B"], c["G"], c["H"], c["T"], c["op"]
    mean_t = T - (T // 2) / 2.0 * (B - 1) / B if c["ragged"] else T
    bg = B * G
    row = KV4_ROW if c["fmt"] == "kv4" else BF16_ROW
    if op == "prompt":
        # keys and values read, the cache written, its values written
        return dict(bytes=bg * mean_t * 2 * (BF16_ROW + KV4_ROW + BF16_ROW), flops=bg * mean_t * 2 * D * 6)
    if op == "append":
        # the token in, its row out, and (where the window completes) 31 keys; one block of values
        tail = min(T, 32)
        return dict(bytes=bg * 2 * (BF16_ROW + KV4_ROW + tail * (KV4_ROW + BF16_ROW)), flops=bg * 2 * tail * D * 2)
    if op in ("attend", "mass"):
        blocks = (mean_t + BLOCK - 1) // BLOCK
        tokens = mean_t if c["topk"] == 0 else min(mean_t, min(c["topk"] + 2, blocks) * BLOCK)
        idx = 0 if c["topk"] == 0 else bg * (c["topk"] + 3) * 4
        mass = 8 * bg * min(c["topk"] + 2, blocks) if op == "mass" else 0
        return dict(bytes=bg * tokens * 2 * row + 2 * bg * H * BF16_ROW + idx + mass, flops=bg * H * tokens * D * 4)
    blocks = min(c["keep"], (mean_t + BLOCK - 1) // BLOCK)
    tokens = min(mean_t, c["keep"] * BLOCK)
    b = bg * tokens * 2 * row * 2 + bg * blocks * 4 * BF16_ROW * 2 + bg * 4 * (mean_t / BLOCK + 2 * c["keep"])
    if c["fmt"] == "kv4":
        b += bg * tokens * 2 * BF16_ROW
    return dict(bytes=b, flops=bg * blocks * 32 * D)


# ------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The same outputs from the definitions in 64 bits. The stored 4-bit values are defined by
    roundings (of scale, zero, code and value), which are part of the definition."""
    global own
    kept_own, own = own, False
    try:
        raw = _raw_inputs(case, seed)
    finally:
        own = kept_own
    op, c = raw["op"], case
    if op == "prompt":
        live = (torch.arange(raw["cap"], device="cuda")[None] < raw["seq"].long()[:, None])[:, None, :, None]
        zero = torch.zeros((), dtype=torch.float64, device="cuda")
        return dict(k=torch.where(live, _grid64(raw["k"], torch.bfloat16), zero),
                    v=torch.where(live, _grid64(raw["v"], torch.float16), zero))
    if op == "append":
        return _exact_append(raw)
    if op == "evict":
        return _exact_evict(raw, c)
    k, v = raw["k"], raw["v"]
    if c["fmt"] == "kv4":
        k, v = _grid64(k, torch.bfloat16), _grid64(v, torch.float16)
    B, G, H, nb = c["B"], c["G"], c["H"], raw["nb"]
    q = raw["q"].double().reshape(B * G, H, D)
    hit = torch.ones((B, G, nb), dtype=torch.bool, device="cuda")
    if c["topk"]:
        hit = torch.zeros((B, G, nb + 1), dtype=torch.bool, device="cuda")
        hit.scatter_(2, torch.where(raw["idx"] >= 0, raw["idx"], torch.full_like(raw["idx"], nb)).long(), True)
        hit = hit[..., :nb]
    outs, masses = [], []
    for n in range(B * G):               # one sequence-group at a time: the scores are large in 64 bits
        b, g = divmod(n, G)
        t = torch.arange(raw["cap"], device="cuda")
        on = hit[b, g][t // BLOCK] & (t < raw["seq"][b])
        at = on.nonzero()[:, 0]
        kk, vv = k[b, g][at].double(), v[b, g][at].double()
        logits = q[n] @ kk.T / D**0.5
        e = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
        e = e / e.sum(dim=1, keepdim=True)
        outs.append(e @ vv)
        masses.append(torch.zeros(nb, dtype=torch.float64, device="cuda").index_add_(0, at // BLOCK, e.sum(dim=0)))
    out = torch.stack(outs).reshape(B, G * H, D)
    if op == "attend":
        return dict(out=out)
    return dict(out=out, mass=raw["mass"].double() + torch.stack(masses).reshape(B, G, nb))


def _exact_append(raw):
    """The compressed keys after the append: the mean of the completed window's stored values."""
    B, G = raw["B"], raw["G"]
    ck = raw["ck"].double().clone()
    for b, t in enumerate(raw["seq"].tolist()):
        if t >= 32 and t % 16 == 0:
            keys = torch.cat((raw["k"][b, :, t - 32 : t - 1], raw["k_new"][b][:, None]), dim=1)
            ck[b, :, (t - 32) // 16] = _grid64(keys, torch.bfloat16).mean(dim=1)
    at = (raw["seq"].long() - 1) % BLOCK
    k, v = torch.zeros((2, B, G, 3, BLOCK, D), dtype=torch.float64, device="cuda")
    for b, t in enumerate(raw["seq"].tolist()):
        first = (t - 1) // BLOCK * BLOCK
        for out, old, new, dtype in ((k, raw["k"], raw["k_new"], torch.bfloat16), (v, raw["v"], raw["v_new"], torch.float16)):
            out[b, :, 0, : at[b]] = _grid64(old[b, :, first : t - 1], dtype)
            out[b, :, 0, at[b]] = _grid64(new[b], dtype)
    return dict(k=k, v=v, ck=ck)


def _exact_evict(raw, c):
    """The compressed keys of the kept blocks (everything else is moved, not computed)."""
    keep, recent = c["keep"], c["recent"]
    ck = torch.zeros_like(raw["dst_ck"], dtype=torch.float64)
    for b, t in enumerate(raw["seq"].tolist()):
        n = (t + BLOCK - 1) // BLOCK
        for g in range(c["G"]):
            m = raw["mass"][b, g, :n].tolist()
            fixed = {0} | set(range(max(0, n - recent), n))
            rest = sorted((j for j in range(n) if j not in fixed), key=lambda j: (-m[j], j))
            blocks = sorted(fixed | set(rest[: max(0, keep - len(fixed))]))
            rows, at = [], []
            for i, j in enumerate(blocks):
                left = t - BLOCK * (n - len(blocks)) - BLOCK * i
                for w in range(4):
                    if 16 * w + 32 <= left:
                        rows.append((4 * j + w, i, w < 3 or (i + 1 < len(blocks) and blocks[i + 1] == j + 1)))
                        at.append(4 * i + w)
            if not rows:
                continue
            src = torch.tensor([r if same else 0 for r, _, same in rows], device="cuda")
            got = raw["ck"][b, g][src].double()
            new = [(x, i) for x, (_, i, same) in enumerate(rows) if not same]
            if new:
                tail = torch.tensor([[blocks[i] * BLOCK + 48 + u for u in range(16)] + [blocks[i + 1] * BLOCK + u for u in range(16)] for _, i in new], device="cuda")
                keys = raw["k"][b, g][tail]
                keys = _grid64(keys, torch.bfloat16) if c["fmt"] == "kv4" else keys.double()
                got[torch.tensor([x for x, _ in new], device="cuda")] = keys.mean(dim=1)
            ck[b, g, torch.tensor(at, device="cuda")] = got
    return dict(k=None, v=None, ck=ck, kept=None, mass=None, seq_len=None)


def _raw_inputs(case, seed):
    """prepare()'s inputs with the keys and values still in bf16."""
    return prepare(dict(case, fmt="bf16"), seed)


def _grid64(x, dtype):
    """Each value of x [..., 128] replaced by the value that its 4-bit code stands for, float64."""
    shape = x.shape
    x = x.double().reshape(-1, GROUP)
    lo, hi = x.min(dim=1, keepdim=True).values, x.max(dim=1, keepdim=True).values
    step = ((hi - lo).float() / 15.0).to(dtype).double()
    base = (lo - 16.0 * step).float().to(dtype).double()
    steps = (x - base).float().double() / step
    level = torch.round(steps - 16.0).clamp(0.0, 15.0)
    level = torch.where(step > 0, level, torch.zeros_like(level))
    x = step * (16.0 + level)
    x += base
    return x.to(dtype).double().reshape(shape)
